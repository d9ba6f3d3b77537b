"""Host-side refusals of the head norms and rotation, and what the binding hands over
(no GPU needed)."""
import ctypes

import pytest
import torch

from libutil import ensure_built

NULL, SHAPE, ALIGN, DTYPE, ALIAS = 1, 2, 4, 5, 7
# addresses that are never followed, far from one another
Q, K, QO, KO, WQ, WK, T, P = ((i + 1) << 36 for i in range(8))


@pytest.fixture(scope="module")
def w4():
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    return mod


def call(w4, **change):
    a = dict(q=Q, qo=QO, qs=1024, qos=1024, wq=WQ, hq=8, k=K, ko=KO, ks=256, kos=256, wk=WK, hk=2, t=T,
             rows=100, rot=128, il=0, eps=1e-6, p=P, n=50, d=128, dt=1, no_q=False, no_k=False, no_how=False)
    a.update(change)
    q = w4._HeadRowsStruct(a["q"], a["qo"], a["qs"], a["qos"], a["wq"], a["hq"])
    k = w4._HeadRowsStruct(a["k"], a["ko"], a["ks"], a["kos"], a["wk"], a["hk"])
    how = w4._NormRopeStruct(a["t"], a["rows"], a["rot"], a["il"], a["eps"])
    at = lambda s, none: None if none else ctypes.addressof(s)  # noqa: E731
    return w4.lib().w4_qk_norm_rope(at(q, a["no_q"]), at(k, a["no_k"]), at(how, a["no_how"]), a["p"],
                                    a["n"], a["d"], a["dt"], None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), DTYPE), (dict(no_how=True), NULL), (dict(no_q=True, no_k=True), NULL),
    (dict(t=None, wq=None, wk=None), NULL), (dict(t=None, wq=None, no_k=True), NULL),
    (dict(d=96), SHAPE), (dict(d=256), SHAPE), (dict(n=-1), SHAPE), (dict(n=(1 << 24) + 1), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(rows=0), SHAPE), (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE),
    (dict(il=2), SHAPE), (dict(hq=0), SHAPE), (dict(hk=1025), SHAPE), (dict(qs=1016), SHAPE),
    (dict(qs=1028), SHAPE), (dict(kos=248), SHAPE), (dict(q=None), NULL), (dict(ko=None), NULL),
    (dict(p=None), NULL), (dict(q=Q + 8), ALIGN), (dict(ko=KO + 2), ALIGN), (dict(wk=WK + 4), ALIGN),
    (dict(t=T + 8), ALIGN), (dict(p=P + 2), ALIGN), (dict(n=0, q=None, k=None, p=None), 0),
])
def test_refusals(w4, change, status):
    assert call(w4, **change) == status


@pytest.mark.parametrize("change", [
    dict(qo=Q + 2048), dict(qo=Q, qos=2048), dict(qo=K), dict(ko=QO + 512, kos=1024), dict(ko=QO + 2048),
    dict(qo=T + 4096), dict(ko=P), dict(qo=WQ), dict(qo=WK), dict(ko=WQ),
    # slices of one buffer of 14 heads (3584 bytes a row) that share columns
    dict(q=Q, qo=Q, qs=1792, qos=1792, k=Q + 2048 - 256, ko=Q + 2048 - 256, ks=1792, kos=1792),
    # out of place, but onto the other side's input
    dict(q=Q, qs=1792, k=Q + 2048, ks=1792, qo=Q + 1024, qos=1792),
    # keys whose row of the buffer runs into the next token's queries
    dict(q=Q, qo=Q, qs=1792, qos=1792, k=Q + 3584 - 256, ko=Q + 3584 - 256, ks=1792, kos=1792),
])
def test_outputs_that_share_bytes_are_refused(w4, change):
    assert call(w4, **change) == ALIAS


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be followed")
@pytest.mark.parametrize("change", [
    dict(), dict(qo=Q, ko=K),
    dict(q=Q, qo=Q, qs=1792, qos=1792, k=Q + 2048, ko=Q + 2048, ks=1792, kos=1792),      # in place
    dict(q=Q, qo=Q, qs=1792, qos=1792, k=Q + 2048 - 3584, ko=Q + 2048 - 3584, ks=1792, kos=1792),
    dict(q=Q, k=Q + 2048, qs=1792, ks=1792),                                              # to new rows
    dict(q=Q, k=Q + 2048, qs=1792, ks=1792, qo=QO, ko=QO + 2048, qos=1792, kos=1792),
    dict(no_k=True, qo=K), dict(no_q=True, p=None, t=None), dict(wq=None, wk=None), dict(qs=1 << 30, n=1),
])
def test_accepted(w4, change):
    """As far as the check of the device, which is the last."""
    assert call(w4, **change) in (8, 9)


def test_binding_refusals(w4):
    x = torch.zeros((3, 6, 64), dtype=torch.bfloat16)
    pos, table, w = torch.zeros(3, dtype=torch.int32), torch.ones((10, 64)), torch.ones(64)
    bad = [dict(q=None, k=None), dict(q=x[0]), dict(k=x[:2]), dict(k=x.half()), dict(k=x[..., :32]),
           dict(q=x.float(), k=None), dict(table=table.double()), dict(table=table[:, ::2]),
           dict(table=table[:0]), dict(table=table[0]), dict(positions=pos[:2]),
           dict(positions=pos.long()), dict(q_weight=w.bfloat16()), dict(q_weight=torch.ones(32)),
           dict(k_weight=torch.ones(128)[::2]), dict(q_out=x[:, :2]), dict(k_out=x.half()),
           dict(q=x.transpose(0, 1).contiguous().transpose(0, 1))]
    seen = []
    real = w4._one_gpu
    w4._one_gpu = lambda *_: None  # the tensors here are not on a GPU
    try:
        for change in bad:
            args = dict(q=x, k=x.clone(), positions=pos, table=table, q_weight=w, k_weight=w)
            args.update(change)
            with pytest.raises(ValueError):
                seen.append(w4.qk_norm_rope(**args))
    finally:
        w4._one_gpu = real
    assert not seen
    with pytest.raises(ValueError):  # on the CPU
        w4.qk_norm_rope(x, x.clone(), pos, table, w, w)


def test_status_string(w4):
    assert "POSITION" in w4.w4_status_string(17)
