"""Decayed linear attention on the GPU against the recurrence in 64 bits: kda_lin_chunk_fwd and
kda_lin_recurrent_step over types, head layouts, ragged lengths, segments, checkpoints, extreme decays, idle
rows, streams and graphs."""
import pytest
import torch

import kda_linear_attention_02_b200 as kda
import lin_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def make(lens, Hqk, H, dk, dv, dtype, decay="token", init=True, seed=0):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    T = sum(lens)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)).to(dtype)  # noqa: E731
    la = {"token": lambda: -torch.exp(1.2 * r(T, H) - 3.0), "fast": lambda: -torch.exp(1.5 * r(T, H) + 1.0),
          "head": lambda: -torch.exp(r(H) - 3.0)}[decay]()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return dict(q=unit(r(T, Hqk, dk)), k=unit(r(T, Hqk, dk)), v=r(T, H, dv).to(dtype), la=la,
                init=0.3 * r(len(lens), H, dk, dv) if init else None, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))


def outputs(x, stride=0):
    T, H, dv = x["v"].shape
    n, dk = x["cu"].numel() - 1, x["q"].shape[2]
    ckcu = kda.kda_ckpt_offsets(x["cu"].cpu(), stride).to(DEV) if stride else None
    nan = lambda *s, dtype=F32: torch.full(s, float("nan"), dtype=dtype, device=DEV)  # noqa: E731
    return dict(o=nan(T, H, dv, dtype=x["v"].dtype), fs=nan(n, H, dk, dv), ckcu=ckcu,
                ck=nan(int(ckcu[-1]), H, dk, dv) if stride else None)


def call(x, y, stride=0, **kw):
    kda.kda_lin_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["init"], x["cu"], y["o"], y["fs"], ckpt_stride=stride,
                          checkpoints=y["ck"], ckpt_cu=y["ckcu"], **kw)
    return y


def verify(x, y, stride=0):
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    o, b, fs, afs, ck, ack = ref.run(x["q"], x["k"], x["v"], x["la"], x["cu"], x["init"], stride)
    cu = x["cu"].tolist()
    longest, dk = max(v - u for u, v in zip(cu, cu[1:])), x["q"].shape[2]
    f = ref.f32_factor(longest, dk)
    if o.numel():
        ref.check("o", y["o"], o, ref.o_tolerance(o, b, y["o"].dtype, longest, dk))
    ref.check("final_state", y["fs"], fs, f * afs + 1e-30)
    if stride and ck.numel():
        ref.check("checkpoints", y["ck"], ck, f * ack + 1e-30)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1], [64], [63, 65, 0, 1, 130, 32, 31, 33, 200]], ids=["one", "chunk", "ragged"])
def test_chunk_shapes(dtype, dk, dv, lens):
    x = make(lens, 2, 2, dk, dv, dtype)
    verify(x, call(x, outputs(x)))


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("decay", ["token", "fast"])
def test_a_single_chunk_rounds_o_once(dk, dv, decay):
    # From a zero state o is made of the scores alone, which keep 16 bits (two bf16 parts: half a step of the second
    # is 2^-8 of what the first left, at most 2^-8).  The exponents are differences of sums of logarithms, each off by
    # at most seven roundings (six additions of a scan and a product): 14 half steps of the largest sum.  What is left
    # is o's own rounding, half a bf16 step.
    lens = [1, 2, 3, 5, 64, 33, 1]
    x = make(lens, 1, 2, dk, dv, BF, decay, init=False, seed=12)
    y = call(x, outputs(x))
    torch.cuda.synchronize()
    o, b = ref.run(x["q"], x["k"], x["v"], x["la"], x["cu"], None)[:2]
    g = max(float(s.sum(0).abs().max()) for s in x["la"].clamp_min(ref.LOG_MIN).split(lens))
    tol = (2.0 ** -16 + ref.f32_factor(64, dk) + 14 * g * 2.0 ** -24) * b * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-30
    ref.check("o", y["o"], o, tol)


def test_stores_ahead_of_ragged_ends():
    # pairs that end in a ragged chunk, which writes o without a tile store, several for each CTA
    x = make([129, 191, 65, 130, 257, 70] * 8, 8, 8, 128, 128, BF, init=False, seed=13)
    verify(x, call(x, outputs(x)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hqk,H", [(1, 1), (1, 6), (3, 6)])
@pytest.mark.parametrize("decay", ["token", "fast", "head"])
def test_chunk_heads_and_decays(dtype, Hqk, H, decay):
    x = make([100, 7, 300], Hqk, H, 128, 64, dtype, decay, init=decay != "token", seed=1)
    verify(x, call(x, outputs(x)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("stride", [64, 192, 512])
def test_chunk_checkpoints(dtype, stride):
    x = make([700, 64, 0, 63, 513], 2, 4, 128, 128, dtype, seed=2)
    verify(x, call(x, outputs(x, stride), stride), stride)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 64), (F32, 64, 128)], ids=["bf16", "bf16-64", "f32"])
@pytest.mark.parametrize("init", [False, True])
def test_chunk_long_sequences_run_in_segments(dtype, dk, dv, init):
    # one sequence of several segments beside short ones, checkpoints across the boundaries
    x = make([5, 3333, 1500, 0, 1], 1, 2, dk, dv, dtype, init=init, seed=3)
    verify(x, call(x, outputs(x, 512), 512), 512)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_short_sequences_beside_a_long_one(dtype):
    # more sequences than one block takes in a round, so that segments are not ordered by length
    lens = [(7 * i) % 4 for i in range(2500)]
    lens[1200] = 1300
    x = make(lens, 1, 2, 64, 64, dtype, seed=14)
    verify(x, call(x, outputs(x)))


def test_calls_on_two_streams_at_once():
    xs = [make([2100, 64, 1], 2, 4, 128, 128, BF, seed=20), make([900, 33] * 6, 4, 4, 64, 128, BF, "fast", seed=21),
          make([1500, 7], 2, 2, 128, 64, F32, seed=22)]
    want = [call(x, outputs(x)) for x in xs]
    got = [[outputs(x) for x in xs] for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for ys in got:
        for x, y, s in zip(xs, ys, streams):
            call(x, y, stream=s)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    for ys in got:
        for y, w in zip(ys, want):
            assert torch.equal(y["o"], w["o"]) and torch.equal(y["fs"], w["fs"])


def test_resume_from_a_checkpoint():
    x = make([1000], 2, 4, 128, 128, BF, seed=4)
    full = call(x, outputs(x, 512), 512)
    tail = {**x, **{n: x[n][512:].contiguous() for n in ("q", "k", "v", "la")}, "init": full["ck"][:1].contiguous(),
            "cu": torch.tensor([0, 488], dtype=torch.int32, device=DEV)}
    y = call(tail, outputs(tail))
    torch.cuda.synchronize()
    assert torch.equal(y["o"], full["o"][512:]) and torch.equal(y["fs"], full["fs"])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_decays_that_forget(dtype):
    # minus infinity, NaN, the lowest value and everything under -120 are a decay of 0; 0 keeps all
    x = make([150, 90], 1, 2, 64, 64, dtype, seed=5)
    la = x["la"]
    la[3], la[64], la[65], la[100] = float("-inf"), float("nan"), torch.finfo(F32).min, -1e4
    la[149, 0], la[150], la[200:210] = -121.0, float("-inf"), 0.0
    verify(x, call(x, outputs(x)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_stay_in_their_sequence(dtype, bad):
    x = make([70, 65, 64, 33], 2, 2, 128, 128, dtype, seed=6)
    want = call(x, outputs(x))
    y = {**x, **{n: x[n].clone() for n in ("q", "k", "v", "init")}}
    for n in ("q", "k", "v"):
        y[n][70:135] = bad              # the whole of sequence 1, whose rows lie behind the others' tails
    y["init"][1] = bad
    got = call(y, outputs(y))
    torch.cuda.synchronize()
    for s in (slice(0, 70), slice(135, None)):
        assert torch.equal(got["o"][s], want["o"][s])
    for i in (0, 2, 3):
        assert torch.equal(got["fs"][i], want["fs"][i])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_earlier_chunks_and_other_heads_ignore_a_nan(dtype):
    x = make([300], 2, 2, 128, 128, dtype, seed=7)
    want = call(x, outputs(x))
    y = {**x, "v": x["v"].clone()}
    y["v"][200, 1] = float("nan")
    got = call(y, outputs(y))
    torch.cuda.synchronize()
    assert torch.equal(got["o"][:192], want["o"][:192]) and torch.equal(got["o"][:, 0], want["o"][:, 0])
    assert torch.equal(got["fs"][:, 0], want["fs"][:, 0]) and got["o"][200:, 1].isnan().all()


def test_empty_batches():
    x = make([0, 0], 1, 2, 64, 64, BF, seed=8)
    y = call(x, outputs(x))
    torch.cuda.synchronize()
    assert torch.equal(y["fs"], x["init"])
    x["init"] = None
    y = call(x, outputs(x))
    torch.cuda.synchronize()
    assert not y["fs"].any()
    x = make([], 1, 2, 64, 64, BF, init=False)
    call(x, outputs(x))


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99]])
def test_bad_sequence_tables_write_nothing(cu):
    x = make([40, 20, 40], 1, 2, 64, 64, BF)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y = call(x, outputs(x))
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == -7
    assert y["o"].isnan().all() and y["fs"].isnan().all()


def test_checkpoints_over_the_states_are_refused():
    x = make([200, 200], 1, 1, 64, 64, BF)
    pool = torch.zeros(8, 1, 64, 64, device=DEV)
    y = outputs(x, 64)
    y["ck"] = pool[:6]
    for name, a, b in (("initial_state", pool[5:7], y["fs"]), ("final_state", x["init"], pool[5:7])):
        x["init"], y["fs"] = a, b
        with pytest.raises(ValueError, match=name):
            call(x, y, 64)


def test_bad_checkpoint_table_is_reported():
    x = make([200, 200], 1, 1, 64, 64, BF)
    y = outputs(x, 64)
    y["ckcu"] = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)   # room for 2 of sequence 0's 3 checkpoints
    call(x, y, 64)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == -7
    assert y["ck"][5].isnan().all() and not y["ck"][:5].isnan().any()


def test_chunk_repeats_bit_for_bit_on_another_stream_and_in_graphs():
    x = make([900, 1, 2100, 64], 2, 4, 128, 128, BF, "fast", seed=9)
    want = call(x, outputs(x, 64), 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(x, outputs(x, 64), 64, stream=s)
    s.synchronize()
    same = lambda a, b: all(torch.equal(a[n], b[n]) for n in ("o", "fs", "ck"))  # noqa: E731
    assert same(got, want)
    ws = torch.full((kda.kda_lin_chunk_fwd_workspace_bytes(3065, 4, 4, 128, 128),), 255, dtype=torch.uint8, device=DEV)
    out = [outputs(x, 64), outputs(x, 64)]
    graphs = []
    with torch.cuda.stream(s):
        for y in out:   # two graphs that share a workspace, replayed in one stream's order
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call(x, y, 64, workspace=ws)
            graphs.append(g)
        for _ in range(2):
            for g in graphs:
                g.replay()
    s.synchronize()
    assert same(out[0], want) and same(out[1], want)
    assert kda.kda_get_device_status() == 0


# ------------------------------------------------------------------------------------------------ step


def step_inputs(n, Hqk, H, dk, dv, dtype, pool, decay="token", seed=0):
    x = make([1] * n, Hqk, H, dk, dv, dtype, decay, init=False, seed=seed)
    g = torch.Generator(DEV)
    g.manual_seed(seed + 100)
    x["state"] = torch.randn(pool, H, dk, dv, generator=g, device=DEV)
    x["o"] = torch.full((n, H, dv), float("nan"), dtype=dtype, device=DEV)
    return x


def step_reference(x, slots):
    live = [i for i, s in enumerate(slots) if s >= 0]
    cu = torch.arange(len(live) + 1)
    la = x["la"] if x["la"].dim() == 1 else x["la"][live]
    return live, ref.run(x["q"][live], x["k"][live], x["v"][live], la, cu, x["state"][[slots[i] for i in live]])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("n,Hqk,H,decay", [(1, 1, 1, "head"), (5, 2, 4, "token"), (300, 1, 2, "fast")])
def test_step(dtype, dk, dv, n, Hqk, H, decay):
    x = step_inputs(n, Hqk, H, dk, dv, dtype, n + 3, decay)
    slots = [(i * 7 + 2) % (n + 3) for i in range(n)] if (n + 3) % 7 else list(range(n))
    if n > 1:
        slots[-1] = slots[1] = -1      # idle rows, within the batch and at its end
    live, (o, b, fs, afs, _, _) = step_reference(x, slots)
    before = x["state"].clone()
    kda.kda_lin_recurrent_step(x["state"], x["q"], x["k"], x["v"], x["la"], x["o"],
                               slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    tol = ref.f32_factor(1, dk) * b + 1e-30 + (2.0 ** -8 * o.abs() if dtype == BF else 0)   # one rounding of o
    ref.check("o", x["o"][live], o, tol)
    used = [slots[i] for i in live]
    ref.check("state", x["state"][used], fs, ref.f32_factor(1, dk) * afs + 1e-30)
    rest = [s for s in range(n + 3) if s not in used]
    assert torch.equal(x["state"][rest], before[rest])
    idle = [i for i in range(n) if slots[i] < 0]
    assert x["o"][idle].isnan().all()


def test_step_without_slots_and_with_a_table_column():
    x = step_inputs(6, 2, 2, 64, 128, BF, 6, seed=3)
    table = torch.full((6, 5), -7, dtype=torch.int32, device=DEV)
    table[:, 2] = torch.arange(6, device=DEV)
    outs, states = [], []
    for slots in (None, table[:, 2]):
        s, o = x["state"].clone(), x["o"].clone()
        kda.kda_lin_recurrent_step(s, x["q"], x["k"], x["v"], x["la"], o, slots=slots)
        outs.append(o)
        states.append(s)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and torch.equal(*states) and not outs[0].isnan().any()


def test_step_leaves_out_rows_with_bad_or_shared_slots():
    x = step_inputs(5, 1, 2, 64, 64, BF, 4, seed=4)
    before = x["state"].clone()
    kda.kda_lin_recurrent_step(x["state"], x["q"], x["k"], x["v"], x["la"], x["o"],
                               slots=torch.tensor([1, 0, 1, 4, 2], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == -7
    assert torch.equal(x["state"][[1, 3]], before[[1, 3]]) and x["o"][[0, 2, 3]].isnan().all()
    assert not torch.equal(x["state"][0], before[0]) and not x["o"][[1, 4]].isnan().any()


def test_step_forgets_and_ignores_what_is_idle():
    x = step_inputs(3, 1, 1, 64, 64, F32, 3, seed=5)
    x["la"][:] = torch.tensor([[float("-inf")], [float("nan")], [0.0]], device=DEV)
    x["q"][2] = x["k"][2] = x["v"][2] = x["la"][2] = float("nan")       # an idle row's inputs
    kda.kda_lin_recurrent_step(x["state"], x["q"], x["k"], x["v"], x["la"], x["o"],
                               slots=torch.tensor([0, 2, -1], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for i, s in ((0, 0), (1, 2)):
        assert torch.equal(x["state"][s, 0], torch.outer(x["k"][i, 0], x["v"][i, 0]))


def test_steps_follow_a_prompt_and_match_the_chunked_form():
    # a prompt, then single tokens from its state: the whole sequence's recurrence, token by token
    for dtype in (BF, F32):
        x = make([90], 1, 2, 128, 128, dtype, seed=11)
        head = {**x, **{n: x[n][:70].contiguous() for n in ("q", "k", "v", "la")},
                "cu": torch.tensor([0, 70], dtype=torch.int32, device=DEV)}
        y = call(head, outputs(head))
        full = outputs(x)
        full["o"][:70] = y["o"]
        state = y["fs"]
        for t in range(70, 90):
            kda.kda_lin_recurrent_step(state, *(x[n][t:t + 1].contiguous() for n in ("q", "k", "v", "la")), full["o"][t:t + 1])
        full["fs"] = state
        verify(x, full)


def test_step_in_a_graph():
    x = step_inputs(4, 1, 2, 128, 128, BF, 4, seed=6)
    want, o = x["state"].clone(), x["o"].clone()
    for _ in range(3):
        kda.kda_lin_recurrent_step(want, x["q"], x["k"], x["v"], x["la"], o)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        kda.kda_lin_recurrent_step(x["state"], x["q"], x["k"], x["v"], x["la"], x["o"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x["state"], want) and torch.equal(x["o"], o)


@pytest.mark.slow
def test_states_beyond_32_bit_offsets():
    # a pool whose last states lie behind 2^32 elements (17 GB) and a batch behind 2^31 bytes
    H, d = 32, 128
    pool = torch.zeros((1 << 32) // (H * d * d) + 2, H, d, d, device=DEV)
    x = step_inputs(2, 1, H, d, d, BF, 2, seed=7)
    small, o = x["state"].clone(), x["o"].clone()
    last = pool.shape[0] - 1
    pool[last], pool[last - 1] = small[0], small[1]
    kda.kda_lin_recurrent_step(small, x["q"], x["k"], x["v"], x["la"], o)
    kda.kda_lin_recurrent_step(pool, x["q"], x["k"], x["v"], x["la"], x["o"],
                               slots=torch.tensor([last, last - 1], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(pool[last], small[0]) and torch.equal(pool[last - 1], small[1]) and torch.equal(x["o"], o)
    assert not pool[:2].any()
