"""How many bits the bf16 chunks of the decayed linear attention keep, against the recurrence in 64 bits."""
import pytest
import torch

import kda_linear_attention_02_b200 as kda
import lin_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def chunk(q, k, v, la, cu, init=None, stride=0):
    """(o, final states, checkpoints) of a call that has to end well."""
    T, H, dv = v.shape
    n, dk = cu.numel() - 1, q.shape[2]
    ckcu = kda.kda_ckpt_offsets(cu.cpu(), stride).to(DEV) if stride else None
    o = torch.full((T, H, dv), float("nan"), dtype=v.dtype, device=DEV)
    fs = torch.full((n, H, dk, dv), float("nan"), device=DEV)
    ck = torch.full((int(ckcu[-1]), H, dk, dv), float("nan"), device=DEV) if stride else None
    kda.kda_lin_chunk_fwd(q, k, v, la, init, cu, o, fs, ckpt_stride=stride, checkpoints=ck, ckpt_cu=ckcu)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    return o, fs, ck


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("resets", [0, 1, 8, 24, 31, 40, 56])
@pytest.mark.parametrize("reset", [-100.0, float("-inf")])
def test_scores_behind_forgotten_tokens_keep_their_bits(dk, dv, resets, reset):
    # Some tokens at a chunk's start forget everything, the rest forget little.  q and k are unit vectors of one
    # channel, so that every score is exactly 1 and a weight is the decay alone; two tokens behind the resets have
    # values of opposite sign, so that o is the small difference of two weights and its own rounding hides nothing.
    # A weight e^x, x >= -120, comes from an exponent that two roundings put off by at most 2 x 120 x 2^-24 < 2^-16,
    # and is kept in two bf16 parts, 2^-8 of 2^-8; the rest is a few half steps of fp32 (the exponential two, the
    # sums of two products one each).
    H, n = 8, 64
    g = torch.Generator(DEV)
    g.manual_seed(resets)
    la = -torch.exp(1.5 * torch.randn(2 * n, H, generator=g, device=DEV) - 6.0)
    la[:resets], la[n:n + resets] = reset, reset
    q = torch.zeros(2 * n, 1, dk, dtype=BF, device=DEV)
    q[..., 3] = 1.0
    v = torch.zeros(2 * n, H, dv, dtype=BF, device=DEV)
    u = (1.0 + torch.rand(dv, generator=g, device=DEV)).to(BF)
    for h in range(H):      # another pair for each head, in both sequences
        i, j = resets + h * (n - 3 - resets) // H, resets + 1 + h * (n - 3 - resets) // H + h % 2
        v[i, h], v[j, h], v[n + i, h], v[n + j, h] = u, -u, -u, u
    cu = ints([0, n, 2 * n])
    o, fs, _ = chunk(q, q, v, la, cu)
    want, b, ws, aws, _, _ = ref.run(q, q, v, la, cu, None)
    ref.check("o", o, want, (2.0 ** -16 + 2.0 ** -16 + 2.0 ** -20) * b + 2.0 ** -8 * want.abs() + 1e-30)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_results_depend_on_the_batch_through_its_tokens_alone(dtype):
    # a long sequence that is cut into segments, at the same place in batches of as many tokens, other sequences beside it
    H, d = 2, 64
    g = torch.Generator(DEV)
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    T = 100 + 3000 + 500
    q, k, v, la = (0.1 * r(T, 1, d)).to(dtype), (0.1 * r(T, 1, d)).to(dtype), r(T, H, d).to(dtype), -0.05 * r(T, H).abs()
    init = r(2, H, d, d)
    got = []
    for lens in ([100, 3000, 500], [100, 3000, 1, 0, 299, 200], [60, 40, 3000, 500]):
        at = lens.index(3000)
        cu = ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s0 = torch.zeros(len(lens), H, d, d, device=DEV)
        s0[at] = init[0]
        # what the others hold must not matter either
        rest = torch.cat([torch.arange(100), torch.arange(3100, T)]).to(DEV)
        x = v.clone()
        x[rest] = r(rest.numel(), H, d).to(dtype)
        o, fs, _ = chunk(q, k, x, la, cu, s0)
        got.append((o[100:3100], fs[at]))
    for o, fs in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(fs, got[0][1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,stride", [(64, 0), (61, 0), (330, 64), (3000, 512)], ids=["chunk", "ragged", "chunks", "segments"])
def test_what_a_token_leaves_in_the_state_is_exact_to_fp32(dtype, dk, dv, T, stride):
    # One token of each head has a value, so that the state is the single product w k v, w the decay up to its chunk's end
    # (nothing decays in other chunks, whose factors are exactly 1, and adding zeros is exact).  With w exact to
    # 2^-22 (the exponential) and the logarithms' sum to a rounding of at most 4 in magnitude (4 x 2^-24), two roundings
    # of the products and one of the sum, that is 2^-22 + 7 x 2^-24 of the value: bf16 has to have all of w v's 24 bits.
    H, n = 16, 3
    g = torch.Generator(DEV)
    g.manual_seed(T + dk + dv)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v = (r(n * T, 1, dk)).to(dtype), (r(n * T, 1, dk)).to(dtype), torch.zeros(n * T, H, dv, dtype=dtype, device=DEV)
    la, cu = torch.zeros(n * T, H, device=DEV), ints([0, T, 2 * T, 3 * T])
    for i in range(n):
        for h in range(H):
            j = ((i * H + h) * 1009 + h) % T if i else min(T - 1, 4 * h)           # all over; in the first, a chunk's places
            c = j - j % 64
            e = min(T, c + 64)
            v[i * T + j, h] = r(dv).to(dtype)
            la[i * T + c:i * T + e, h] = -0.06 * torch.rand(e - c, generator=g, device=DEV)
    _, fs, ck = chunk(q, k, v, la, cu, stride=stride)
    _, _, want, _, wck, _ = ref.run(q, k, v, la, cu, None, stride)
    bound = 2.0 ** -22 + 7 * 2.0 ** -24
    ref.check("final_state", fs, want, bound * want.abs())
    if stride:
        # (the checkpoint at a chunk's end, and those behind it)
        ref.check("checkpoints", ck, wck, bound * wck.abs())
    assert (want != 0).any(dim=(2, 3)).all()


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("decay", [-6.0, -1.0, 1.0])
def test_scores_keep_their_second_part_in_every_chunk(dk, dv, decay):
    # Every chunk's first token forgets what was before, so that o is made of its chunk's scores alone: in every chunk,
    # of sequences of several and of pairs that a CTA takes one behind another.  Scores: two bf16 parts (2^-16), the
    # exponent (2^-16, above), fp32 sums; then o's own rounding.
    lens = [64, 130, 1, 200, 63, 65, 128, 7] * 3
    T, H = sum(lens), 16
    g = torch.Generator(DEV)
    g.manual_seed(dk + dv)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(BF)  # noqa: E731
    q, k, v, la = unit(r(T, 2, dk)), unit(r(T, 2, dk)), r(T, H, dv).to(BF), -torch.exp(r(T, H) + decay)
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    for a, b in zip(starts, starts[1:]):
        la[a:b:64] = float("-inf")
    o, _, _ = chunk(q, k, v, la, ints(starts), 0.3 * r(len(lens), H, dk, dv))
    want, b = ref.run(q, k, v, la, ints(starts), None)[:2]
    tol = (2.0 ** -16 + 2.0 ** -16 + ref.f32_factor(64, dk)) * b * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 1e-30
    ref.check("o", o, want, tol)
    # with one part, the half step of 2^-8 that this would leave in each score shows where values cancel
    assert float((2.0 ** -8 * b / tol).max()) > 20
