"""The append's launch for calls larger than L2 keeps (two heads a thread, reads
and writes past L2): sets of heads that hold a query and a key, a key and a value,
or one head behind the last, rows that are skipped, queries in place, keys alone.

Tolerances as of test_gpu_kv: exact to fp32 before the one rounding."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, _lib, _spx, i32, near, pools, rotate  # noqa: E402,F401

pytestmark = pytest.mark.gpu
LARGE = 64 << 20  # bytes read and written from which on the launch takes two heads a thread


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,heads,kv,P,interleaved,norms,order,page", [
    (128, 7, 3, 128, False, True, "token", 64), (128, 8, 3, 64, True, False, "head", 16), (128, 5, 2, 0, False, True, "joint", 48),
    (64, 7, 4, 64, False, True, "outer", 32), (64, 4, 1, 16, True, True, "token", 16), (64, 9, 9, 32, False, False, "head", 64)])
def test_append_of_many_rows(D, heads, kv, P, interleaved, norms, order, page, dtype):
    spx, g = _spx(), torch.Generator(device="cuda").manual_seed(D + heads)
    # (over the border without the queries too, for the call of keys alone)
    B, n = 5, LARGE // (4 * 2 * kv * D) + 3
    assert 4 * n * 2 * kv * D >= LARGE
    per = -(-(n // B + 2) // page)
    k, v = pools(B * per + 1, page, kv, D, dtype, order)
    k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    table = torch.randperm(B * per + 1, generator=g, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    cache = spx.KvCache(k, v, table, i32([per * page] * B))
    qkv = torch.randn(n, heads + 2 * kv, D, generator=g, device="cuda").to(dtype)
    at = torch.randperm(n, generator=g, device="cuda")  # a place of its own for each row
    req, slot = (at % B).to(torch.int32), (at // B).to(torch.int32)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda").to(torch.int32)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)) if norms else (None, None)
    angle = torch.arange(5000, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, max(P, 1), 2, device="cuda") / max(P, 1))
    cos, sin = (angle.cos().float().contiguous(), angle.sin().float().contiguous()) if P else (None, None)
    # rows that are skipped, of a block's last and first lanes among them, and the last row
    slot[0], slot[31], slot[n - 1], pos[5], pos[64], req[9], req[10], slot[11] = -1, -5, -1, -3, 5000 if P else -1, -1, B, per * page
    live = (slot >= 0) & (pos >= 0) & (pos < 5000 if P else pos >= 0)
    table[1, per // 2] = -1
    stored = live & (req >= 0) & (req < B) & (slot < per * page) & ~((req == 1) & (slot // page == per // 2))
    assert int((~live).sum()) >= 5 and int((live & ~stored).sum()) >= 3 + page // 2
    want_q, want_k = qkv[:, :heads].double(), qkv[:, heads:heads + kv].double()
    for y, w in ((want_q, wq), (want_k, wk)):
        if w is not None:
            y /= (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            y *= w.double()
    if P:
        turn = pos.clamp(0, 4999).long()
        want_q, want_k = (rotate(y, cos[turn], sin[turn], interleaved) for y in (want_q, want_k))
    where = (table[req.clamp(0, B - 1).long(), (slot.clamp(0, per * page - 1) // page).long()].long()[stored],
             (slot % page).long()[stored])
    changed = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    changed[where] = True
    before_k, before_v, raw = k.clone(), v.clone(), qkv.clone()
    q_out = torch.full((n, heads + 1, D), 7.0, dtype=dtype, device="cuda")

    def append(**kw):
        k.copy_(before_k)
        v.copy_(before_v)
        args, keep = spx.kv_append_args(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], req, slot, pos=pos, k_norm=wk,
                                        cos=cos, sin=sin, interleaved=interleaved, **kw)
        spx.spx_kv_append(args)
        assert near(k[where], want_k[stored], dtype) and torch.equal(v[where], raw[stored][:, heads + kv:])
        assert torch.equal(k[~changed], before_k[~changed]) and torch.equal(v[~changed], before_v[~changed])

    append(q=qkv[:, :heads], q_out=q_out[:, :heads], q_norm=wq)
    assert near(q_out[live][:, :heads], want_q[live], dtype)
    assert (q_out[~live] == 7).all() and (q_out[:, heads] == 7).all() and torch.equal(qkv, raw)
    keys = k[where]
    append(q=qkv[:, :heads], q_norm=wq)  # in place
    assert torch.equal(qkv[live][:, :heads], q_out[live][:, :heads]) and torch.equal(qkv[~live], raw[~live])
    assert torch.equal(qkv[:, heads:], raw[:, heads:]) and torch.equal(k[where], keys)
    append()  # keys and values alone
    assert torch.equal(k[where], keys)


def test_both_launches_agree():
    """A call above the border and the same rows in calls below it: the same bits."""
    spx, g = _spx(), torch.Generator(device="cuda").manual_seed(4)
    D, heads, kv, dtype = 128, 6, 3, BF16
    n = LARGE // (4 * (heads + 2 * kv) * D) + 1
    k, v = (torch.full((-(-n // 64), 64, kv, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    cache = spx.KvCache(k, v, torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None].contiguous(), i32([n]))
    qkv = torch.randn(n, heads + 2 * kv, D, generator=g, device="cuda").to(dtype)
    req, slot = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    angle = torch.arange(n, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    cos, sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()

    def append(rows):
        q_out = torch.empty(rows.stop - rows.start, heads, D, dtype=dtype, device="cuda")
        x = qkv[rows]
        args, keep = spx.kv_append_args(cache, x[:, heads:heads + kv], x[:, heads + kv:], req[rows], slot[rows], q=x[:, :heads],
                                        q_out=q_out, q_norm=w, k_norm=w, cos=cos, sin=sin)
        spx.spx_kv_append(args)
        return q_out

    whole = append(slice(0, n))
    keys, values = k.clone(), v.clone()
    k.fill_(math.nan)
    v.fill_(math.nan)
    assert torch.equal(torch.cat([append(slice(0, n // 2)), append(slice(n // 2, n))]), whole)
    for now, then in ((k, keys), (v, values)):
        assert torch.equal(now.flatten(0, 1)[:n], then.flatten(0, 1)[:n])
