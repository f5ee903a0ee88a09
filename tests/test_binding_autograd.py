"""dispatch and combine have gradients, as calls of their own, but record no graph: tensors that
require a gradient are refused where a graph is being recorded, so that none is lost unseen."""
import pytest
import torch

import q4_routed_expert_amd as q4

bf16 = torch.bfloat16


def tensors(**wants):
    r = q4.DeviceRouting(3, 8, 2, "cpu")
    t = {"x": torch.zeros(3, 128, dtype=bf16), "rows": torch.zeros(6, 128, dtype=bf16),
         "base": torch.zeros(3, 128, dtype=bf16)}
    for name in wants:
        if name == "topk_w":  # as a copy into it leaves it
            r.topk_w.copy_(torch.ones_like(r.topk_w).requires_grad_())
        else:
            t[name].requires_grad_()
    return t, r


def calls(t, r):
    return {"x": lambda: q4.dispatch(t["x"], r), "x8": lambda: q4.dispatch(t["x"], r, e4m3=True),
            "rows": lambda: q4.combine(t["rows"], r), "base": lambda: q4.combine(t["rows"], r, base=t["base"]),
            "plain": lambda: q4.combine(t["rows"], r, weighted=False)}


@pytest.mark.parametrize("wants,refused", [("x", {"x", "x8"}), ("rows", {"rows", "base", "plain"}),
                                           ("base", {"base"}), ("topk_w", {"rows", "base"})])
def test_a_graph_is_not_cut(wants, refused):
    t, r = tensors(**{wants: True})
    for name, call in calls(t, r).items():
        # (without a GPU the call that is taken ends at its tensors' device)
        with pytest.raises(ValueError, match="no graph" if name in refused else "on the GPU"):
            call()
    for off in (torch.no_grad, torch.inference_mode):
        for call in calls(t, r).values():
            with off(), pytest.raises(ValueError, match="on the GPU"):
                call()


def test_a_function_of_torch_may_call_them():
    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, r):
            return q4.combine(rows, r)

    t, r = tensors(rows=True)
    with pytest.raises(ValueError, match="on the GPU"):
        Combine.apply(t["rows"], r)
