"""A layer's training operators far out, so that a tile, a row or an element lost there shows: every tile of the longest text,
without a window and with windows, and clipping and rotation behind 2^31 elements."""
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, make_context

pytestmark = pytest.mark.gpu

B = torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def matched(n, window, seed):
    """One head of a text of n rows.  Every tile of 128 has one key of length 8, every tile one query that points to two or three
    of these keys, and all other keys are short: the matched ones have most of the query's sum.  Returns qkv, do and the rows of
    those queries and keys."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q, k, v, do = normal(n, 64), 0.1 * normal(n, 64), normal(n, 64) + 0.5, normal(n, 64) + 0.5
    tiles = torch.arange(n // 128, device="cuda")
    special = normal(len(tiles), 64)
    special *= 8 / special.norm(dim=1, keepdim=True)
    if 0 <= window < 128:         # as far from two keys as the window allows
        at_key, at_query, shifts = 128 * tiles + 74 - window, 128 * tiles + 74, (0, 1)
    else:
        at_key = 128 * tiles + torch.randint(0, 128, (len(tiles),), generator=g, device="cuda")
        at_query = 128 * tiles + torch.randint(0, 128, (len(tiles),), generator=g, device="cuda")
        shifts = (0, 337, 701) if window < 0 else (0, 13, window // 128 - 2)
    k[at_key] = special
    aim = torch.zeros_like(special)
    for s in shifts:
        aim += special.roll(-s, 0)
    q[at_query] = 1.75 * aim
    return torch.cat([q, k, v], 1).to(B), do.to(B), at_query, at_key


@pytest.mark.parametrize("window", [-1, 64, 5000])
def test_every_tile_of_the_longest_text(enc, window):
    n = 131072
    qkv, do, at_query, at_key = matched(n, window, 1)
    cu = lu.offsets([n])
    o, lse, _ = lu.attention_forward(enc, qkv, cu, 1, window)
    g = lu.attention_backward(enc, qkv, cu, o, lse, do, 1, window)
    assert enc.device_status() == binding.TEE_OK
    q, k, v = qkv.double().view(n, 3, 64).unbind(1)
    d, stat = do.double(), lse[0].double()
    delta, delta_size = (d * o.double()).sum(1), (d * o.double()).abs().sum(1)

    def scores(rows, cols):
        """Scores of query rows with key columns, what they are off by, and P of the log sums that the operator has."""
        s, size = q[rows] @ k[cols].t() / 8, q[rows].abs() @ k[cols].abs().t() / 8
        if window >= 0:
            s.masked_fill_((rows[:, None] - cols).abs() > window, -torch.inf)
        p = torch.exp(s - stat[rows, None])
        off = lu.mma(64, size) + 2.0 ** -22 * (size + 2 * stat[rows, None].abs() + 1)
        return s, p, off

    def gradient(rows, cols):
        """dS and P of rows and columns, and what they are off by as the products' operands."""
        _, p, off = scores(rows, cols)
        dp, dp_size = d[rows] @ v[cols].t(), d[rows].abs() @ v[cols].abs().t()
        ds = p * (dp - delta[rows, None])
        ds_off = 1.01 * (p * (lu.mma(64, dp_size) + 2.0 ** -20 * delta_size[rows, None]) + ds.abs() * off)
        return ds, ds_off + lu.HALF * (ds.abs() + ds_off), p, 1.01 * p * (off + lu.HALF)

    def close(got, w, w_off, other, lost, scale=1.0):
        """got against scale w other, w's rows off by w_off; each row's largest term is seen to matter."""
        want, size = scale * (w @ other), scale * (w.abs() @ other.abs())
        off = scale * (w_off @ other.abs()) * 1.01 + lu.mma(n, size)
        bound = off + lu.HALF * (want.abs() + off)
        assert_within(got, want, bound)
        for j in lost:      # without this column's term the row would not be right
            term = scale * w.gather(1, j[:, None]) * other[j]
            seen = (term.abs() > 2 * bound).any(1)
            assert int(seen.sum()) > 0.9 * len(seen), int(seen.sum())

    every = torch.arange(n, device="cuda")
    for part in range(0, len(at_query), 256):
        rows, cols = at_query[part:part + 256], at_key[part:part + 256]
        s, p, off = scores(rows, every)
        # the scores' errors as they weigh in the sum; its logarithm in fp32, and the log sum's own rounding and scale
        assert_within(stat[rows], torch.logsumexp(s, 1), (p * off).sum(1) * 1.01 + 2.0 ** -20 * (1 + stat[rows].abs()))
        close(o[rows], p, 1.01 * p * (off + lu.HALF), v, [p.argmax(1)])
        ds, ds_off, _, _ = gradient(rows, every)
        close(g[rows, :64], ds, ds_off, k, [ds.abs().argmax(1)], 1 / 8)
        ds, ds_off, p, p_off = (x.t().contiguous() for x in gradient(every, cols))
        close(g[cols, 64:128], ds, ds_off, q, [ds.abs().argmax(1)], 1 / 8)
        close(g[cols, 128:], p, p_off, d, [p.argmax(1)])


def test_clipping_behind_two_to_the_31_elements(enc):
    """Scaled and copied, in place and not."""
    n = (1 << 31) + 20001
    flat = torch.zeros(n, dtype=B, device="cuda")
    places = [0, 1 << 30, (1 << 31) - 10000, n - 12000]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    values = [torch.randn(10000, generator=gen, device="cuda").to(B) for _ in places]
    for a, t in zip(places, values):
        flat[a:a + 10000] = t
    want = sum(float(t.double().square().sum()) for t in values) ** 0.5

    def check(out, factor):
        for a, t in zip(places, values):
            assert_within(out[a:a + 10000], t.double() * factor, 2.0 ** -8 * (t.double() * factor).abs())
        ends = [a + 10000 for a in places]
        for a, b in zip([0] + ends, places + [n]):
            assert not bool(out[a:b].any())

    out = torch.full_like(flat, 3.0)
    for max_norm in (1e30, 5.0):
        norm, factor = lu.clip(enc, [flat], max_norm, [out]).tolist()
        assert abs(norm - want) < 2.0 ** -18 * want and abs(factor - min(1, max_norm / want)) <= 2.0 ** -18 * factor
        check(out, factor)
    check(flat, 1.0)
    norm, factor = lu.clip(enc, [flat], 5.0).tolist()
    check(flat, factor)


def test_rotation_behind_two_to_the_31_elements(enc):
    """The last rows of 3.2e9 elements, at the positions of their own text, forward and backward and in place."""
    heads, T, last = 12, 1400000, 320
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    tail = torch.randn(last, 192 * heads, generator=g, device="cuda").to(B)
    pos = (torch.arange(T, device="cuda") - (T - last)).remainder(last).to(torch.int32)
    x = torch.zeros(T, 192 * heads, dtype=B, device="cuda")
    x[-last:] = tail
    for backward in (False, True):
        want = lu.rope(enc, tail, pos[-last:].contiguous(), heads, 160000.0, backward)
        y = lu.rope(enc, x, pos, heads, 160000.0, backward)
        assert torch.equal(y[-last:], want) and not bool(y[:-last].any())
    lu.rope(enc, x, pos, heads, 160000.0, backward, y=x)
    assert torch.equal(x[-last:], want) and not bool(x[:-last].any())
