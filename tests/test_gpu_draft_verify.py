"""GPU parity: draft_verify against oracle/draft.py (rational arithmetic).

Tokens and counts must be equal. The kernel's products and differences are
exact in float64; its running sums are off by at most V 2^-53 relative, so each
case first asserts that its target lies further than V 2^-50 of the total from
every running sum near it (the oracle's own margin)."""

import numpy as np
import pytest
import torch

import int8_hadamard_domain_amd as i8h
from oracle import draft

pytestmark = pytest.mark.gpu


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _case(B, D, V, seed, greedy, dtype, near=0.5):
    rng = np.random.default_rng(seed)
    t = 2.0 * rng.standard_normal((B, D + 1, V))
    d = t[:, :D] + near * rng.standard_normal((B, D, V))
    p = torch.from_numpy(_softmax(t)).to(dtype)
    q = None if greedy else torch.from_numpy(_softmax(d)).to(dtype)
    pick = d if greedy else d + rng.gumbel(size=d.shape)
    x = pick.argmax(-1).astype(np.int32) if D else np.zeros((B, 0), np.int32)
    u = rng.random((B, D), dtype=np.float32)
    un = rng.random(B, dtype=np.float32)
    length = np.minimum(rng.integers(0, 2 * D + 1, B), D).astype(np.int32)
    return p, q, x, length, u, un


def _np(t):
    return None if t is None else t.float().numpy().astype(np.float64)


def _gpu(p, q, x, length, u, un, **kw):
    c = lambda a: None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    tokens, accepted = i8h.draft_verify(c(p), c(q), c(x), c(u), c(un), draft_len=c(length), **kw)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), accepted.cpu().numpy()


def _margin(p, q, x, length, un, accepted):
    """Smallest distance between a target and a running sum, relative to the total, in units of V 2^-50."""
    worst = np.inf
    for b in range(p.shape[0]):
        n, V = accepted[b], p.shape[2]
        row = p[b, n].copy()
        if n < (p.shape[1] - 1 if length is None else length[b]):
            if q is None:
                row[x[b, n]] = 0
            else:
                row = np.maximum(row - q[b, n], 0)
        cum = np.cumsum(row.astype(np.longdouble))
        if cum[-1] > 0:
            worst = min(worst, float(np.abs(cum / cum[-1] - np.longdouble(un[b]))[:-1].min(initial=1.0)) / (V * 2.0 ** -50))
    return worst


CASES = [(1, 0, 1), (1, 1, 2), (3, 4, 7), (2, 15, 100), (1, 15, 4096), (1, 3, 4097), (5, 2, 5000), (2, 15, 8191),
         (8, 15, 1031), (70, 3, 33), (2, 70, 40)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,D,V", CASES)
def test_matches_the_oracle(gpu_available, B, D, V, greedy, dtype):
    print(f"draft_verify B={B} D={D} V={V} greedy={greedy} {dtype}", flush=True)
    p, q, x, length, u, un = _case(B, D, V, B + D + V, greedy, dtype)
    want_t, want_n = draft.verify_batch(_np(p), _np(q), x, length, u, un)
    assert _margin(_np(p), _np(q), x, length, un, want_n) > 1
    got_t, got_n = _gpu(p, q, x, length, u, un)
    assert np.array_equal(got_n, want_n) and np.array_equal(got_t, want_t)
    want_t, want_n = draft.verify_batch(_np(p), _np(q), x, None, u, un)      # no draft_len: D everywhere
    got_t, got_n = _gpu(p, q, x, None, u, un)
    assert np.array_equal(got_n, want_n) and np.array_equal(got_t, want_t)


def test_large_vocabulary(gpu_available):
    """Against float64 running sums (the rational oracle is slow here)."""
    B, D, V = 3, 5, 262144 + 77
    print("draft_verify large vocabulary", flush=True)
    p, q, x, length, u, un = _case(B, D, V, 5, False, torch.float32)
    got_t, got_n = _gpu(p, q, x, length, u, un)
    P, Q = _np(p), _np(q)
    for b in range(B):
        n = 0
        while n < length[b] and float(u[b, n]) * Q[b, n, x[b, n]] < P[b, n, x[b, n]]:
            n += 1
        rest = np.maximum(P[b, n] - Q[b, n], 0) if n < length[b] else P[b, n]
        cum = np.cumsum(rest.astype(np.longdouble))
        nxt = int((cum <= np.longdouble(un[b]) * cum[-1]).sum())
        assert got_n[b] == n and got_t[b].tolist() == x[b, :n].tolist() + [nxt] + [-1] * (D - n)


@pytest.mark.parametrize("V", [5, 4096, 9000])
def test_ends_of_the_range_and_fallbacks(gpu_available, V):
    """u at 0 and just below 1, empty rests, entries that are not probabilities, tokens that are none."""
    print(f"draft_verify edges V={V}", flush=True)
    rng = np.random.default_rng(V)
    B, D = 12, 2
    p = _softmax(rng.standard_normal((B, D + 1, V)))
    q = _softmax(rng.standard_normal((B, D, V)))
    x = rng.integers(0, V, (B, D)).astype(np.int32)
    u = np.zeros((B, D), np.float32)
    top = np.float32(1 - 2.0 ** -24)
    un = np.full(B, 0.5, np.float32)
    un[0], un[1] = 0.0, top
    p[2, 0] = q[2, 0]; u[2, 0] = top; p[2, 0, x[2, 0]] = 0; q[2, 0] = np.maximum(p[2, 0], q[2, 0])  # nothing left of p - q
    p[3, 0] = 0                                              # an empty row
    p[4, 0, 0], p[4, 0, V - 1], x[4, 0] = np.nan, np.inf, 0
    p[5, 0, 1] = -3.0; x[5, 0] = 1
    x[6, 0], x[7, 0] = -1, V
    x[8, 1] = 2 ** 31 - 1
    u[9] = top
    un[10] = 0.0; p[10, 0, :V // 2] = 0; x[10, 0] = 0; q[10, 0, :] = 0; q[10, 0, 0] = 1
    un[11] = top; p[11, 0, V // 2:] = 0; x[11, 0] = V - 1
    with np.errstate(invalid="ignore"):
        for draft_probs in (q, None):
            want_t, want_n = draft.verify_batch(p, draft_probs, x, None, u, un)
            got_t, got_n = _gpu(torch.from_numpy(p), None if draft_probs is None else torch.from_numpy(q), x, None, u, un)
            assert np.array_equal(got_n, want_n)
            assert np.array_equal(got_t, want_t), np.argwhere(got_t != want_t)


def test_draft_len_is_clamped(gpu_available):
    p, q, x, _, u, un = _case(4, 3, 50, 9, False, torch.float32)
    length = np.array([-5, 0, 3, 99], np.int32)
    want = draft.verify_batch(_np(p), _np(q), x, length, u, un)
    got = _gpu(p, q, x, length, u, un)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_no_sequences(gpu_available):
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    t, n = i8h.draft_verify(e(0, 4, 9), e(0, 3, 9), e(0, 3, dt=torch.int32), e(0, 3), e(0))
    assert t.shape == (0, 4) and n.shape == (0,)


# ------------------------------------------------------------------------------------- many chunks, large tensors

def _running(P, Q, x, length, u, un):
    """One sequence against extended-precision running sums."""
    n = 0
    while n < length and float(u[n]) * (1.0 if Q is None else Q[n, x[n]]) < P[n, x[n]]:
        n += 1
    rest = P[n].copy()
    if n < length:
        if Q is None:
            rest[x[n]] = 0
        else:
            rest = np.maximum(rest - Q[n], 0)
    cum = np.cumsum(rest.astype(np.longdouble))
    target = np.longdouble(un) * cum[-1]
    assert np.abs(cum - target).min() > len(rest) * 2.0 ** -50 * cum[-1]
    return n, int((cum <= target).sum())


@pytest.mark.parametrize("B,V,dtype", [(1, 1 << 20, torch.float32), (2, 1100003, torch.float32),
                                       (2, 1100004, torch.bfloat16), (90, 40000, torch.bfloat16),
                                       (300, 8192, torch.float32), (300, 8191, torch.bfloat16)])
@pytest.mark.parametrize("greedy", [False, True])
def test_many_chunks(gpu_available, B, V, dtype, greedy):
    """Rows of more chunks than a workgroup has threads, and batches that take the larger chunks."""
    print(f"draft_verify B={B} V={V} {dtype} greedy={greedy}", flush=True)
    D = 2
    p, q, x, length, u, un = _case(B, D, V, V + B, greedy, dtype)
    un[0] = 0.999
    got_t, got_n = _gpu(p, q, x, length, u, un)
    P, Q = _np(p), _np(q)
    for b in range(0, B, max(1, B // 12)):
        n, nxt = _running(P[b], None if Q is None else Q[b], x[b], length[b], u[b], un[b])
        assert got_n[b] == n and got_t[b].tolist() == x[b, :n].tolist() + [nxt] + [-1] * (D - n)


def test_probabilities_past_2_31_elements(gpu_available):
    """A row that starts past 2^31 elements is found, kept and drawn from."""
    B, D, V = 2, 1023, (1 << 20) + 5
    p = torch.zeros((B, D + 1, V), dtype=torch.bfloat16, device="cuda")
    print("draft_verify past 2^31 elements", flush=True)
    assert p.numel() > 1 << 31
    x = torch.randint(0, V, (B, D), generator=torch.Generator().manual_seed(1)).int()
    x[1, 1000] = 77
    for b in range(B):
        p[b, torch.arange(D, device="cuda"), x[b].long().cuda()] = 1.0
    p[1, 1000, 77] = 0.0                            # refused there
    p[1, 1000, V - 3] = 0.5
    p[0, D, 123456] = 0.25
    p[0, D, 654321] = 0.75
    u, un = np.full((B, D), 0.5, np.float32), np.array([0.3, 0.9], np.float32)
    c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    tokens, accepted = i8h.draft_verify(p, None, x.cuda(), c(u), c(un))
    assert accepted.tolist() == [D, 1000]
    want = torch.cat([x[0], torch.tensor([654321], dtype=torch.int32)])
    assert torch.equal(tokens[0].cpu(), want)
    assert tokens[1].tolist() == x[1, :1000].tolist() + [V - 3] + [-1] * 23


def test_unaligned_rows_and_outputs(gpu_available):
    """Rows at every alignment of their element, outputs inside larger buffers."""
    B, D, V = 3, 2, 1027
    for dtype in (torch.float32, torch.bfloat16):
        print(f"draft_verify unaligned {dtype}", flush=True)
        p, q, x, length, u, un = _case(B, D, V, 31, False, dtype)
        want = draft.verify_batch(_np(p), _np(q), x, length, u, un)
        for shift in (1, 2, 3):
            pb = torch.empty(p.numel() + shift, dtype=dtype, device="cuda")[shift:].view(p.shape)
            pb.copy_(p)
            qb = torch.empty(q.numel() + 4 - shift, dtype=dtype, device="cuda")[4 - shift:].view(q.shape)
            qb.copy_(q)
            tok = torch.full((B + 2, D + 1), 9, dtype=torch.int32, device="cuda")
            acc = torch.full((B + 2,), 9, dtype=torch.int32, device="cuda")
            t, n = _gpu(pb, qb, x, length, u, un, tokens=tok[1:-1], accepted=acc[1:-1])
            assert np.array_equal(n, want[1]) and np.array_equal(t, want[0])
            assert (tok[0] == 9).all() and (tok[-1] == 9).all() and acc[0] == 9 and acc[-1] == 9


@pytest.mark.parametrize("B,chunks,chunk", [(200, 40, 1024), (27, 300, 1024), (300, 40, 4096)])
def test_empty_chunks_at_a_border(gpu_available, B, chunks, chunk):
    """Rows of a few entries (as a top-k filter leaves them), the draw on the border before a run of empty chunks:
    the token holds probability, and the target lies at one of its ends, off by the sums' rounding at most."""
    V = chunks * chunk
    print(f"draft_verify empty chunks B={B} V={V}", flush=True)
    rng = np.random.default_rng(B + chunks)
    p = np.zeros((B, 1, V), np.float32)

    def put(b, c, value):       # 48 bits of it, as two entries of a chunk
        hi = np.float32(value)
        if float(hi) > value:
            hi = np.nextafter(hi, np.float32(0))
        lo = np.float32(value - float(hi))
        p[b, 0, c * chunk + 5], p[b, 0, c * chunk + 77] = hi, lo
        return float(hi) + float(lo)
    for b in range(B):
        total = 0.0
        for c in np.sort(rng.choice(chunks - 12, int(rng.integers(3, 12)), replace=False)):
            total += put(b, c, rng.random() * 2.0 ** -int(rng.integers(0, 30)))
        put(b, chunks - 3, total)      # as much again behind the empty chunks: u_next = 0.5 is the border
    un = np.full(B, 0.5, np.float32)
    tokens, accepted = _gpu(torch.from_numpy(p), None, np.zeros((B, 0), np.int32), None, np.zeros((B, 0), np.float32), un)
    assert not accepted.any()
    for b in range(B):
        row = p[b, 0].astype(np.longdouble)
        run, t = np.cumsum(row), tokens[b, 0]
        target, off = 0.5 * run[-1], V * 2.0 ** -50 * run[-1]
        assert row[t] > 0, (b, t)
        assert run[t] > target - off and run[t] - row[t] <= target + off, (b, t)


@pytest.mark.parametrize("V", [(1 << 31) - 1, (1 << 31) - 1024])
def test_the_largest_vocabularies(gpu_available, V):
    print(f"draft_verify V={V}", flush=True)
    p = torch.zeros((1, 1, V), dtype=torch.bfloat16, device="cuda")
    at = [5, 1 << 30, V - 2, V - 1]
    p[0, 0, torch.tensor(at, device="cuda")] = 0.25
    none = torch.empty((1, 0), device="cuda")
    for i, v in enumerate(at):
        un = torch.tensor([0.25 * i + 0.1], device="cuda")
        tokens, accepted = i8h.draft_verify(p, None, none.int(), none, un)
        assert tokens.tolist() == [[v]] and accepted.tolist() == [0]
