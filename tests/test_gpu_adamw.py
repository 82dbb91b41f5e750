"""AdamW over many tensors, moments in 32 and in 8 bits, against float64."""
import itertools

import pytest
import torch

import adamw64 as plain
import resharding_tensor_parallelism_gb300 as rtp
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LR, BETAS, EPS, DECAY, SEED = 1e-2, (0.9, 0.95), 1e-8, 0.1, 5
# empty, one element, around a lane's 4, a block of 128, a chunk of 1024 and of 4096, and some larger
SIZES = [0, 1, 3, 4, 5, 127, 128, 129, 255, 1023, 1024, 1025, 4095, 4097, 40000]


def _tensors(sizes, dtype, out=None, seed=0, std=1.0, shift=0):
    """Tensors of N(0, std), each `shift` elements behind a 256-byte border."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    got = []
    for n in sizes:
        t = out.empty((n + shift,), dtype)[shift:] if out else torch.empty((n + shift,), dtype=dtype, device="cuda")[shift:]
        got.append(t.copy_(torch.randn(n, generator=gen, device="cuda") * std))
    return got


def _near(got, want, bound, what):
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of the bound" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / bound).max()))


def _moments(group, i):
    n, at = group.params[i].numel(), group.offsets[i]
    m, v = group.exp_avg[at:at + n], group.exp_avg_sq[at:at + n]
    if group.states == 32:
        return m.double(), v.double()
    s = group.scales[at // 128:(at + n + 127) // 128]
    return plain.values(m, s[:, 0], True), plain.values(v, s[:, 1], False)


def _check_step(group, before, grads, t, norm=None, lr=LR):
    """before: (params or masters, m, v) of every tensor ahead of step t."""
    flips = total = 0
    for i, (p, (x, m, v)) in enumerate(zip(group.params, before)):
        n = p.numel()
        if n == 0:
            continue
        new, m1, v1, ep, em, ev = plain.step(x, grads[i].reshape(-1), m, v, t, lr, group.betas, group.eps, group._decay[i],
                                             norm)
        r = plain.noise(n, SEED, i, t, "cuda")
        flat = p.reshape(-1)
        if group.masters[i] is not None:
            _near(group.masters[i].reshape(-1), new, ep, "master %d" % i)
            assert torch.equal(flat, group.masters[i].reshape(-1).to(BF16))
        elif p.dtype is F32:
            _near(flat, new, ep, "param %d" % i)
        else:  # up or down to the neighbours, by 16 random bits; float32 errors may turn values next to a border
            e = torch.frexp(new)[1].clamp(min=-125)
            steps = new.abs() * plain.pow2(8 - e) + (plain.pcg(r) % 65536).double() / 65536
            want = torch.floor(steps) * plain.pow2(e - 8) * torch.sign(new)
            wrong = flat.double() != want
            _near(flat, new, ep + plain.pow2(e - 8), "param %d" % i)
            border = (steps - steps.round()).abs() <= ep * plain.pow2(8 - e) + 2.0 ** -16
            assert not (wrong & ~border).any(), "param %d" % i
        if group.states == 32:
            m_got, v_got = _moments(group, i)
            _near(m_got, m1, em, "m %d" % i)
            _near(v_got, v1, ev, "v %d" % i)
            continue
        at = group.offsets[i]
        scales = group.scales[at // 128:(at + n + 127) // 128].long()
        for name, x1, err, codes, signed, bits, k in (("m", m1, em, group.exp_avg, True, r % 65536, 0),
                                                      ("v", v1, ev, group.exp_avg_sq, False, r // 65536, 1)):
            code, top, near = plain.quantise(x1, (bits.double() + 0.5) / 65536, signed)
            got = codes[at:at + n].long()
            assert (scales[:, k] - top).abs().max() <= 1  # a largest value next to a power of two
            same = (scales[:, k] == top).repeat_interleave(128)[:n]
            if signed:  # codes 0 and 128 both stand for 0: the sign of a sum that cancels is that of its rounding
                got, code = (torch.where(c == 128, 0, c) for c in (got, code))
            wrong = (got != code) & same
            # a code may differ where the fraction is within the float32 error of its border: err, in spacings of at
            # least a 16th of the value (or of the block's smallest spacing)
            spacing = torch.maximum(x1.abs() / 16, plain.pow2(top - 127 - (16 if signed else 32)).repeat_interleave(128)[:n])
            border = near <= 2 * err / spacing + 2.0 ** -19
            for j in torch.nonzero(wrong & ~border)[:1, 0].tolist():
                raise AssertionError("%s of tensor %d, element %d: code %d for %g, %d expected, %g of a spacing from the "
                                     "border, error %g, block exponent %d" % (
                    name, i, j, int(got[j]), float(x1[j]), int(code[j]), float(near[j]), float(err[j]), int(top[j // 128])))
            flips += int(wrong.sum())
            total += n
    assert flips <= 2 + total * 2.0 ** -14


def _before(group):
    return [((p if m is None else m).reshape(-1).double().clone(), *(t.clone() for t in _moments(group, i)))
            for i, (p, m) in enumerate(zip(group.params, group.masters))]


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", F32), ("f32", BF16), ("bf16", F32), ("bf16", BF16), ("master", F32),
                                        ("master", BF16)])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps(states, param, grad, shift):
    out = Guarded()
    params = _tensors(SIZES, F32 if param == "f32" else BF16, out, 1, shift=shift)
    group = rtp.AdamWGroup(params, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, states=states, seed=SEED,
                           masters=True if param == "master" else None)
    for t in range(1, 4):
        grads = _tensors(SIZES, grad, None, 10 + t, 1e-3, shift)
        kept = [g.clone() for g in grads]
        before = _before(group)
        group.step(grads)
        _check_step(group, before, grads, t)
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))
        assert int(group.steps) == t
    out.check("step")


@pytest.mark.parametrize("states", [32, 8])
def test_many_tensors_and_mixed_types(states):
    """600 tensors: more than one launch holds; the small launch holds 32."""
    for n in (31, 33, 257, 600):
        sizes = [1 + (37 * i) % 300 for i in range(n)]
        kinds = list(itertools.islice(itertools.cycle([F32, BF16, BF16]), n))
        params = [t.to(k) for t, k in zip(_tensors(sizes, F32, None, 2), kinds)]
        masters = [p.float() if i % 3 == 2 else None for i, p in enumerate(params)]
        grads = [t.to(k) for t, k in zip(_tensors(sizes, F32, None, 3, 1e-2), kinds[::-1])]
        decay = [0.1 * (i % 2) for i in range(n)]
        group = rtp.AdamWGroup(params, lr=LR, betas=BETAS, weight_decay=decay, states=states, seed=SEED, masters=masters)
        before = _before(group)
        group.step(grads)
        _check_step(group, before, grads, 1)
        assert int(group.steps) == 1


@pytest.mark.parametrize("states", [32, 8])
def test_large_tensors(states):
    """Over 2 x 152 chunks of 4096 elements: four rows a warp."""
    sizes = [3_000_001, 128, 1_500_000]
    params = _tensors(sizes, BF16, None, 4)
    group = rtp.AdamWGroup(params, lr=LR, betas=BETAS, states=states, seed=SEED, masters=True, weight_decay=DECAY)
    for t in (1, 2):
        grads = _tensors(sizes, BF16, None, 20 + t, 1e-3)
        before = _before(group)
        group.step(grads)
        _check_step(group, before, grads, t)


@pytest.mark.parametrize("states", [32, 8])
def test_clipping_by_a_norm_on_the_gpu(states):
    sizes = [1000, 77]
    for std in (1.0, 1e-4):
        params, grads = _tensors(sizes, F32, None, 5), _tensors(sizes, F32, None, 6, std)
        group = rtp.AdamWGroup(params, lr=LR, betas=BETAS, states=states, seed=SEED, weight_decay=DECAY)
        norm = rtp.grad_norm(grads)
        before = _before(group)
        group.step(grads, norm=norm, max_norm=1.0)
        _check_step(group, before, grads, 1, norm)


def test_step_after_clipping_is_the_clipped_step():
    """Clipping in the step does what clip_grad_norm before it does (bf16 gradients are not rounded again)."""
    sizes = [5000, 300]
    grads = _tensors(sizes, F32, None, 7)
    groups = [rtp.AdamWGroup(_tensors(sizes, F32, None, 8), lr=LR, betas=BETAS) for _ in range(2)]
    groups[0].step(grads, norm=rtp.grad_norm(grads), max_norm=0.5)
    norm, clipped = rtp.clip_grad_norm(grads, 0.5, out=[torch.empty_like(g) for g in grads])
    groups[1].step(clipped)
    for a, b in zip(groups[0].params, groups[1].params):
        assert torch.equal(a, b)


def test_learning_rate_on_the_gpu():
    params, grads = _tensors([500], F32, None, 9), _tensors([500], F32, None, 10)
    group = rtp.AdamWGroup(params, lr=1.0, betas=BETAS, seed=SEED, weight_decay=DECAY)
    before = _before(group)
    group.step(grads, lr=torch.tensor(LR, device="cuda"))
    _check_step(group, before, grads, 1)


def test_shapes_and_zero_gradients():
    """Weights of any shape; a first step without a gradient only decays."""
    p = torch.randn((7, 3, 11), device="cuda")
    for states in (32, 8):
        q = p.clone()
        group = rtp.AdamWGroup([q], lr=0.5, weight_decay=0.5, states=states)
        group.step([torch.zeros_like(q)])
        assert torch.allclose(q, p * 0.75, rtol=1e-6) and not any(t.any() for t in group.moments())


@pytest.mark.parametrize("states", [32, 8])
def test_nan_and_infinite_gradients(states):
    """They spoil their own element (8 bits: their block's moments), and nothing else."""
    p = torch.randn(1000, device="cuda")
    g = torch.randn(1000, device="cuda")
    g[300], g[700] = float("nan"), float("inf")
    q = p.clone()
    group = rtp.AdamWGroup([q], lr=LR, states=states)
    group.step([g])
    assert torch.isnan(q[300]) and int(torch.isfinite(q).sum()) >= 998
    m, v = group.moments()
    bad = 1000 if states == 32 else 128
    for t in (m[:1000], v[:1000]):
        wrong = torch.nonzero(~torch.isfinite(t))[:, 0].tolist()
        assert set(wrong) == ({300, 700} if states == 32 else set(range(256, 384)) | set(range(640, 768))), bad


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_of_8_bit_moments(dtype):
    """Every code under several exponents, NaN and the least one among them."""
    group = rtp.AdamWGroup([torch.zeros(7 * 256, device="cuda")], states=8)
    group.exp_avg.copy_(torch.arange(256, dtype=torch.uint8, device="cuda").repeat(7))
    group.exp_avg_sq.copy_(group.exp_avg)
    tops = torch.tensor([0, 0, 27, 27, 100, 100, 127, 127, 128, 128, 200, 200, 255, 255], dtype=torch.uint8, device="cuda")
    group.scales.copy_(torch.stack([tops, tops], 1))
    m, v = group.moments(dtype)
    assert m.dtype is dtype
    for got, codes, signed in ((m, group.exp_avg, True), (v, group.exp_avg_sq, False)):
        want = plain.values(codes, tops, signed)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got.double()[fine], want[fine])


def test_random_rounding_keeps_small_steps():
    """bf16 weights of 1 that move by a 64th of their spacing a step: their mean moves as it should (nearest would not)."""
    n, steps = 1 << 18, 8
    p = torch.ones(n, dtype=BF16, device="cuda")
    group = rtp.AdamWGroup([p], lr=2.0 ** -14, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0, seed=SEED)
    for _ in range(steps):
        group.step([torch.ones(n, dtype=BF16, device="cuda")])  # m / sqrt(v) = 1
    # below 1 the spacing is 2^-8: the sum of n independent roundings deviates by 2^-8 sqrt(n p (1 - p)), p = steps / 64
    sigma = 2.0 ** -8 * (steps / 64) ** 0.5 / n ** 0.5
    assert abs(float(p.double().mean()) - (1 - steps * 2.0 ** -14)) < 6 * sigma


def test_8_bit_second_moments_follow_the_gradients():
    """v of a constant gradient rises to it, although a step changes it by less than half a spacing."""
    n = 1 << 16
    group = rtp.AdamWGroup([torch.zeros(n, device="cuda")], betas=(0.9, 0.99), states=8, seed=SEED)
    for t in range(300):
        group.step([torch.ones(n, device="cuda")])
    want = 1 - 0.99 ** 300
    m, v = group.moments(F32)
    # steps of v: 1 % of the distance, rounded to spacings of an 8th at most, so a variance of under (v / 8)^2 / 4 a step,
    # forgotten over 50 steps: under 0.2 of a value, and of the mean of n values n^-1/2 of that
    assert abs(float(v.double().mean()) - want) < 6 * 0.45 / n ** 0.5
    assert abs(float(m.double().mean()) - 1) < 6 * 0.45 / n ** 0.5


def test_steps_are_reproducible_and_seeds_differ():
    def run(seed, states):
        group = rtp.AdamWGroup(_tensors([5000], BF16, None, 11), states=states, seed=seed, lr=1e-3)
        for t in range(3):
            group.step(_tensors([5000], BF16, None, 30 + t))
        return torch.cat([group.params[0].float(), *(x.float() for x in group.moments())])
    for states in (32, 8):
        a, b, c = run(1, states), run(1, states), run(2, states)
        assert torch.equal(a, b) and not torch.equal(a, c)


@pytest.mark.parametrize("states", [32, 8])
def test_state_travels(states):
    """A group that loads another's state goes on as that one does."""
    sizes = [700, 33]
    a = rtp.AdamWGroup(_tensors(sizes, BF16, None, 12), states=states, seed=3, masters=True)
    for t in range(2):
        a.step(_tensors(sizes, F32, None, 40 + t))
    b = rtp.AdamWGroup([p.clone() for p in a.params], states=states, seed=3, masters=[m.clone() for m in a.masters])
    b.load_state_dict({k: v if isinstance(v, int) else v.clone() for k, v in a.state_dict().items()})
    for group in (a, b):
        group.step(_tensors(sizes, F32, None, 50))
    assert int(b.steps) == 3
    for x, y in zip([*a.params, *a.masters, *a.moments()], [*b.params, *b.masters, *b.moments()]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("states", [32, 8])
def test_captured_steps_count_on(states):
    """Two graphs on one group, replayed in turn: as many steps as replays, with the gradients of the moment."""
    sizes = [3000, 17]
    groups = [rtp.AdamWGroup(_tensors(sizes, BF16, None, 13), states=states, seed=3, lr=1e-3) for _ in range(2)]
    grads = _tensors(sizes, F32, None, 60)
    lr = torch.tensor(1e-3, device="cuda")
    groups[0].step(grads, lr=lr)
    groups[1].step(grads, lr=lr)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            groups[0].step(grads, lr=lr)
    assert int(groups[0].steps) == 1
    for i in range(4):
        for g, new in zip(grads, _tensors(sizes, F32, None, 70 + i)):
            g.copy_(new)
        lr.fill_(1e-3 / (i + 1))
        graphs[i % 2].replay()
        groups[1].step(grads, lr=lr)
    assert int(groups[0].steps) == int(groups[1].steps) == 5
    for x, y in zip([*groups[0].params, *groups[0].moments()], [*groups[1].params, *groups[1].moments()]):
        assert torch.equal(x, y)


def test_another_stream_waits_for_the_groups_state():
    s = torch.cuda.Stream()
    sizes = [2_000_000]
    params, grads = _tensors(sizes, F32, None, 14), _tensors(sizes, F32, None, 15)
    torch.cuda.synchronize()
    for _ in range(3):
        p = [t.clone() for t in params]
        torch.cuda.synchronize()
        junk = torch.full((2_000_000,), float("nan"), device="cuda")  # what the state's memory may hold before
        del junk
        group = rtp.AdamWGroup(p, lr=LR, betas=BETAS, weight_decay=DECAY, seed=SEED)
        before = [(params[0].double(), torch.zeros_like(params[0]).double(), torch.zeros_like(params[0]).double())]
        group.step(grads, stream=s)
        s.synchronize()
        _check_step(group, before, grads, 1)


def test_a_gradients_storage_may_change_between_steps():
    p, g = _tensors([300], F32, None, 16), _tensors([300], F32, None, 17)
    group = rtp.AdamWGroup(p, lr=LR, betas=BETAS, weight_decay=DECAY, seed=SEED)
    group.step(g)
    p[0].data = p[0].data.clone()  # the weight's too
    before = _before(group)
    new = _tensors([300], BF16, None, 18)
    group.step(new)
    _check_step(group, before, new, 2)


def test_refusals():
    p, g = [torch.zeros(8, device="cuda"), torch.zeros(8, dtype=BF16, device="cuda")], torch.zeros(8, device="cuda")
    group = rtp.AdamWGroup(p)
    kept = [t.clone() for t in p]
    for call in (lambda: group.step([g]), lambda: group.step([g, g[:4]]), lambda: group.step([g, g.cpu()]),
                 lambda: group.step([g, torch.zeros(16, device="cuda")[::2]]), lambda: group.step([g, None]),
                 lambda: group.step([g, g], norm=torch.zeros(2, device="cuda")), lambda: group.step([g, g], lr=-1.0),
                 lambda: group.step([g, g], lr=float("nan")), lambda: group.step([g, g], norm=g[0], max_norm=-1.0),
                 lambda: rtp.AdamWGroup([p[0], p[0]]).step([g, g]), lambda: rtp.AdamWGroup([p[0], p[0][4:]]).step([g, g[4:]]),
                 lambda: rtp.AdamWGroup(p, states=16), lambda: rtp.AdamWGroup(p, betas=(1.0, 0.9)),
                 lambda: rtp.AdamWGroup(p, weight_decay=[0.1]), lambda: rtp.AdamWGroup(p, masters=[None]),
                 lambda: rtp.AdamWGroup(p, masters=[g, None]), lambda: rtp.AdamWGroup([p[0].cpu()]),
                 lambda: rtp.AdamWGroup(p, weight_decay=-1.0).step([g, g]),
                 lambda: group.load_state_dict({"step": 1}),
                 lambda: group.load_state_dict({**group.state_dict(), "exp_avg": group.exp_avg[:4]})):
        with pytest.raises(rtp.RtpError):
            call()
    with pytest.raises(TypeError):
        group.step([g, g.double()])
    assert int(group.steps) == 0 and all(torch.equal(a, b) for a, b in zip(p, kept))


def test_an_empty_group_counts_its_steps():
    group = rtp.AdamWGroup([])
    group.step([])
    assert int(group.steps) == 1 and group.moments()[0].numel() == 0
    group = rtp.AdamWGroup([torch.zeros((0, 4), device="cuda")], states=8)
    group.step([torch.zeros((0, 4), device="cuda")])
    assert int(group.steps) == 1 and group.moments()[0].numel() == 0


@pytest.mark.parametrize("n", [1, 130, 5000])
def test_8_bit_moments_anywhere_in_memory(n):
    """Codes and scales at odd places, through the C ABI: as those at whole vectors."""
    def run(shift):
        (p,), (g,) = _tensors([n], F32, None, 20), _tensors([n], F32, None, 21, 1e-3)
        out = Guarded()
        m, v = (out.empty((n + shift,), torch.uint8)[shift:].zero_() for _ in range(2))
        scales = out.empty((2 * ((n + 127) // 128) + 2 * shift,), torch.uint8)[2 * shift:].zero_()
        clock = torch.zeros(16, dtype=torch.int64, device="cuda")
        rtp._check(rtp.lib().rtp_adamw_clock(clock.data_ptr(), 0, 0.9, 0.95, None))
        t = (rtp.AdamWTensor * 1)()
        t[0].numel, t[0].param, t[0].grad, t[0].exp_avg, t[0].exp_avg_sq = n, p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr()
        t[0].scales, t[0].weight_decay = scales.data_ptr(), DECAY
        for _ in range(3):
            rtp._check(rtp.lib().rtp_adamw_step(1, t, 8, LR, None, EPS, None, 1.0, SEED, clock.data_ptr(), None))
        out.check("step")
        return p, m, v, scales
    torch.cuda.synchronize()
    a, b = run(0), run(1)
    assert all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))
    # the two forms of the quotient: each within 2^-20 of itself, of an update of lr at most 3 times over
    assert ((a[0] - b[0]).abs() <= 3 * LR * 2.0 ** -18 + 4 * plain.EPS * a[0].abs()).all()


@pytest.mark.parametrize("top", [1e-12, 1.0, 1e10, 1e30])
def test_8_bit_moments_of_any_size(top):
    """Blocks whose exponents fit the fast form and not, and both in one tensor."""
    n = 4096
    for spread in (1.0, 1e-4):  # squares stay normal float32 numbers
        p, g = _tensors([n], F32, None, 22), _tensors([n], F32, None, 23)
        g[0] *= top ** 0.5 if top > 1 else top
        g[0][::2048] *= spread
        group = rtp.AdamWGroup(p, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, states=8, seed=SEED)
        for t in range(1, 4):
            before = _before(group)
            group.step(g)
            _check_step(group, before, g, t)


def test_two_groups_at_once():
    """Steps of two groups on two streams beside each other."""
    def make(i):
        return rtp.AdamWGroup(_tensors([300_000, 77], BF16, None, 24 + i), lr=LR, states=8 if i else 32, masters=True, seed=SEED)
    grads = [_tensors([300_000, 77], F32, None, 26 + i, 1e-3) for i in range(2)]
    want = [make(i) for i in range(2)]
    for i, group in enumerate(want):
        for _ in range(6):
            group.step(grads[i])
    got, streams = [make(i) for i in range(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, group in enumerate(got):
            group.step(grads[i], stream=streams[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert int(b.steps) == 6
        assert all(torch.equal(x, y) for x, y in zip([*a.params, *a.masters, *a.moments()], [*b.params, *b.masters, *b.moments()]))


def _trained(states, mixed, seed=50):
    sizes = [700, 33, 1]
    params = _tensors(sizes, BF16, None, seed)
    if mixed:
        params[1] = params[1].float()
    group = rtp.AdamWGroup(params, lr=1e-5, states=states, seed=3, masters=True)  # steps far below a bf16 spacing
    for t in range(2):
        group.step(_tensors(sizes, F32, None, seed + 1 + t))
    return group, sizes


def _alike(a, b):
    for x, y in zip([*a.params, *(m for m in a.masters if m is not None), *a.moments()],
                    [*b.params, *(m for m in b.masters if m is not None), *b.moments()]):
        assert torch.equal(x, y)
    assert int(a.steps) == int(b.steps)


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("states", [32, 8])
def test_a_state_holds_the_copies_that_the_group_made(states, mixed):
    """Weights and state_dict are all that goes from one group to another, or back into the same one."""
    a, sizes = _trained(states, mixed)
    weights = [p.clone() for p in a.params]
    state = {k: v if isinstance(v, int) else v.clone() for k, v in a.state_dict().items()}
    b = rtp.AdamWGroup([p.clone() for p in weights], lr=1e-5, states=states, seed=3, masters=True)
    b.load_state_dict({k: v if isinstance(v, int) else v.cpu() for k, v in state.items()})
    _alike(a, b)
    grads = _tensors(sizes, F32, None, 60)
    for group in (a, b):
        group.step(grads)
    _alike(a, b)
    for p, w in zip(a.params, weights):  # back to the saved point
        p.copy_(w)
    a.load_state_dict(state)
    a.step(grads)
    _alike(a, b)


def test_states_whose_copies_do_not_fit_are_refused():
    a, sizes = _trained(32, False)
    state = a.state_dict()
    without = {k: v for k, v in state.items() if k != "masters"}
    plain_group = rtp.AdamWGroup([p.clone() for p in a.params])
    for group, bad in ((a, without), (a, {**state, "masters": state["masters"][:5]}),
                       (a, {**state, "masters": state["masters"].to(BF16)}), (plain_group, state)):
        kept = [t.clone() for t in (group.exp_avg, *group.params)]
        with pytest.raises(rtp.RtpError):
            group.load_state_dict(bad)
        assert all(torch.equal(x, y) for x, y in zip(kept, (group.exp_avg, *group.params)))
    # copies that the caller gave are the caller's own: in no state, and brought up to one that has them
    own = [m.clone() for m in a.masters]
    given = rtp.AdamWGroup([p.clone() for p in a.params], masters=own)
    assert set(given.state_dict()) == {"step", "exp_avg", "exp_avg_sq"}
    given.load_state_dict(without)
    for m in own:
        m.zero_()
    given.load_state_dict(state)
    assert all(torch.equal(x, y) for x, y in zip(own, a.masters))


def test_a_state_waits_for_steps_on_every_stream():
    params = [torch.zeros(50_000_000, device="cuda")]
    group = rtp.AdamWGroup(params, states=8)
    grads = [torch.ones_like(params[0])]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        group.step(grads, stream=s)
    assert group.state_dict()["step"] == 20


def test_tensors_that_are_not_what_the_group_was_built_over():
    """More or fewer tensors than the group's table holds, and copies of another type, are refused; a copy that is gone is
    not written."""
    make = lambda: rtp.AdamWGroup(_tensors([64, 9], BF16, None, 70), masters=True, lr=LR)
    grads = _tensors([64, 9, 5], F32, None, 71)
    for change, n in ((lambda g: (g.params.append(grads[2].clone()), g.masters.append(None)), 3),
                      (lambda g: g.params.append(grads[2].clone()), 3),
                      (lambda g: (g.params.pop(), g.masters.pop()), 1), (lambda g: g.masters.pop(), 2),
                      (lambda g: g.masters.__setitem__(0, g.masters[0].to(BF16)), 2),
                      (lambda g: g.masters.__setitem__(0, None), 1)):
        group = make()
        change(group)
        kept = [p.clone() for p in group.params]
        with pytest.raises(rtp.RtpError):
            group.step(grads[:n])
        assert int(group.steps) == 0 and all(torch.equal(a, b) for a, b in zip(kept, group.params))
    for lr in (LR, torch.tensor(LR, device="cuda")):
        group = make()
        copy = group.masters[0]
        kept = copy.clone()
        group.masters[0] = None
        group.step(grads[:2], lr=lr)
        assert torch.equal(copy, kept) and int(group.steps) == 1


@pytest.mark.parametrize("size", [1.0, 1e-12, 1e10])
@pytest.mark.parametrize("param", ["f32", "bf16", "master"])
@pytest.mark.parametrize("states", [32, 8])
def test_a_step_does_not_depend_on_the_place_in_memory(states, param, size):
    """Tensors that can be read in vectors and not, bit for bit, whichever form of the quotient their blocks take."""
    def run(shift):
        dtype = F32 if param == "f32" else BF16
        group = rtp.AdamWGroup(_tensors([1, 130, 5000], dtype, None, 80, shift=shift), lr=LR, betas=BETAS, weight_decay=DECAY,
                               states=states, seed=SEED, masters=True if param == "master" else None)
        for t in range(3):
            grads = _tensors([1, 130, 5000], F32, None, 81 + t, 1e-3, shift)
            for g in grads[1:]:
                g[100:200] *= size
            group.step(grads)
        return [*group.params, *(m for m in group.masters if m is not None), *group.moments()]
    assert all(torch.equal(a, b) for a, b in zip(run(0), run(1)))


@pytest.mark.parametrize("param", ["f32", "bf16", "master"])
@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("numel", [100, 5000])
def test_replicas_stay_alike(states, param, numel):
    """Pieces that hold the same (one of them elsewhere in its vectors) and are given the same noise do so after any number of
    steps; with another number they are rounded another way."""
    dtype = F32 if param == "f32" else BF16
    make = lambda kind, seed, std: [_tensors([numel], kind, None, seed, std, shift)[0] for shift in (0, 1, 0)]
    group = rtp.AdamWGroup(make(dtype, 30, 1.0), lr=LR, betas=BETAS, weight_decay=DECAY, states=states, seed=SEED,
                           masters=True if param == "master" else None, noise=[4, 4, 1])
    for t in range(4):
        group.step(make(F32, 31 + t, 1e-2))
    first, same, other = (torch.cat([x.double().reshape(-1) for x in (p, *_moments(group, i))] +
                                    ([] if group.masters[i] is None else [group.masters[i].double()]))
                          for i, p in enumerate(group.params))
    assert torch.equal(first, same)
    assert torch.equal(first, other) == (states == 32 and param != "bf16")


@pytest.mark.parametrize("states", [32, 8])
def test_noise_is_the_tensors_place_by_default(states):
    def run(noise):
        group = rtp.AdamWGroup(_tensors([300, 40], BF16, None, 40), lr=LR, states=states, seed=SEED, noise=noise)
        group.step(_tensors([300, 40], F32, None, 41))
        return [*group.params, *group.moments()]
    a, b, c = run(None), run([0, 1]), run([1, 0])
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not torch.equal(a[0], c[0])


def test_noise_that_is_refused():
    p = [torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")]
    for noise in ([0], [0, 1, 2], [0, -1], [0, 2 ** 31 - 1]):
        with pytest.raises(rtp.RtpError):
            rtp.AdamWGroup(p, noise=noise)
    rtp.AdamWGroup(p, noise=[0, 2 ** 31 - 2]).step([torch.zeros_like(t) for t in p])
