"""The window attention family where it could go wrong unseen: workspaces used again with other
inputs, values and positions at the ends of their ranges, many work items per block.  A
result that is NaN where the reference is finite fails here."""
import numpy as np
import pytest

import test_window as T
from self_attention_backward_gb300 import binding as B

lib = T.lib


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("dtype,algo", T.ALGOS)
def test_backward_uses_this_calls_statistics(lib, dtype, algo, layout):
    """Calls that share a workspace in turn on different inputs give what each gives with one of
    its own, bit for bit: row statistics, inputs and outputs lie at the same addresses every time."""
    torch = T._gpu()
    *cases, spare = [T.Case(dtype, 32, 2, 4, 2, 700, 700, 150, 2, seed=60 + i, layout=layout) for i in range(3)]
    fwd = [c.forward(algo) for c in cases]
    want = [c.backward(*f, algo=algo) for c, f in zip(cases, fwd)]
    torch.cuda.synchronize()
    ins = (*spare.t, *spare.forward(algo))
    ws = B.BwdWorkspace()
    got = []
    for n in range(40):
        for to, t in zip(ins, (*cases[n % 2].t, *fwd[n % 2])):
            to.copy_(t)
        q, k, v, do, o, lse = ins
        got.append(B.win_attn_bwd(q, k, v, o, lse, do, cases[0].scale, 150, 2, workspace=ws, algo=algo))
    B.psa_attn_sync_status()
    for n, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[n % 2], g)), n
