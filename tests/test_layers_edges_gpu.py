"""Edges of the layers beside the mixer on the GPU."""
import numpy as np
import pytest

from tests import layers_ref as R
from tests.test_layers_gpu import _torch, check, dev, host, swa_inputs

pytestmark = pytest.mark.gpu


# -------------------------------------------------- queries that see one key
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,window,sinks", [([1] * 7, 40, 2), ([0, 1, 1, 0, 1], 1, 0), ([1] * 300, 5, 64), ([1, 5, 1, 130, 3], 1, 0),
                                               ([700, 1, 2, 300], 1, 0)])
def test_queries_of_one_key_have_no_gradient(lens, window, sinks, d, dtype):
    """The softmax of one score is 1 whatever the score: dq and dk are exactly 0, dv is the group's dO."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", lens[:8], window, sinks, d, dtype, flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(1, sum(lens), sum(lens), 6, 2, d, dtype, len(lens) + d)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o, lse = kd.swa_fwd(q[0], k[0], v[0], window, sinks, cu_seqlens=cu, return_lse=True)
    g = kd.swa_bwd(q[0], k[0], v[0], o, lse, dO[0], window, sinks, cu_seqlens=cu)
    assert not g["dq"].any() and not g["dk"].any()
    a = 0
    for n in lens:
        s = slice(a, a + n)
        a += n
        if n > 1 or a <= 8:
            val, err = R.attention_heads(qv[0, s], kv[0, s], vv[0, s], window, sinks, 1 / np.sqrt(d), ov[0, s], R.unit(dtype))
            check("dv", g["dv"][s], val["dv"], err["dv"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,window,sinks", [(1, 1, 4, 2, 9, 3), (300, 300, 2, 1, 1, 0), (40, 900, 4, 1, 1, 0),
                                                       (700, 200, 16, 2, 1, 0), (300, 300, 8, 1, 1000, 3), (200, 70, 4, 2, 30, 1)])
def test_queries_of_one_key_in_batches(Tq, Tk, Hq, Hkv, window, sinks, d, dtype):
    """The same batched, also where workgroups share a group's heads; the first query alone where the window is wider,
    an infinity in its value among them (what it sees has no gradient through the softmax)."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", (Tq, Tk, Hq, Hkv, window, sinks, d), dtype, flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(2, Tq, Tk, Hq, Hkv, d, dtype, Tq + Tk + 5 * d)
    o, lse = kd.swa_fwd(q, k, v, window, sinks, return_lse=True)
    g = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks)
    first = Tq - Tk        # the query at position 0
    if first >= 0:
        assert not g["dq"][:, :first + 1].any()
    if window + sinks == 1 or Tk == 1:
        assert not g["dq"].any() and not g["dk"].any()
    for b in range(2):
        val, err = R.attention_heads(qv[b], kv[b], vv[b], window, sinks, 1 / np.sqrt(d), ov[b], R.unit(dtype))
        for n in ("dq", "dk", "dv"):
            check(n, g[n][b], val[n], err[n])


# ------------------------------------------------------- many packed sequences
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,window,sinks", [([3] * 200 + [900] + [7] * 60 + [400] + [1] * 90 + [300, 128, 700], 60, 5),
                                               ([300] * 9, 30, 64), ([187, 188, 189, 0, 0, 600, 1, 188] * 3, 60, 33), ([2600, 200, 1], 1, 1)])
def test_many_packed_sequences_equal_each_alone(lens, window, sinks, dtype):
    """Sequences with queries beyond the window of the first keys among others without; nothing behind the workspace
    is written, nothing in it is read that was not written."""
    import ctypes

    import delta_rule_recurrent_chunk_amd as kd
    from delta_rule_recurrent_chunk_amd import layers as la
    torch = _torch()
    T, Hq, Hkv, d = sum(lens), 4, 2, 64
    print("case", lens[:8], window, sinks, dtype, flush=True)
    (q, _), (k, _), (v, _), (dO, _) = swa_inputs(1, T, T, Hq, Hkv, d, dtype, T)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o, lse = kd.swa_fwd(q[0], k[0], v[0], window, sinks, cu_seqlens=cu, return_lse=True)
    _, desc, *_ = la._swa(q[0], k[0], v[0], window, sinks, None, cu)
    need = kd.lib().kron_delta_swa_workspace_bytes(ctypes.byref(desc), 1)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    g = kd.swa_bwd(q[0], k[0], v[0], o, lse, dO[0], window, sinks, cu_seqlens=cu, workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    a = 0
    for n in lens:
        s = slice(a, a + n)
        a += n
        if n < 100 and a > 200:
            continue
        oo, ll = kd.swa_fwd(q[:, s], k[:, s], v[:, s], window, sinks, return_lse=True)
        gg = kd.swa_bwd(q[:, s], k[:, s], v[:, s], oo, ll, dO[:, s], window, sinks)
        assert torch.equal(o[s], oo[0]) and all(torch.equal(g[m][s], gg[m][0]) for m in g), n
