"""How layer norm, dropout, embedding and cross entropy are called: tensors unlike their
examples, overlaps, neighbours of outputs, graphs, streams, long tables."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import channel_ref as cref
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F32, rand
from tests.test_train_ops_gpu import classes_of, close, d, tokens_of, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def calls(h, rows=80, c=64, v=48):
    """(operator, its right arguments by name, names of its outputs) of every kind."""
    x, r, dy = (rand(rows, c, seed=i, dtype=BF) for i in (1, 2, 3))
    y, t, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    vec, vec2 = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    table, dtable, w = rand(v, c, seed=4, dtype=BF), torch.empty(v, c, dtype=BF, device="cuda"), rand(v, c, seed=5, dtype=BF)
    tokens, target = tokens_of(rows, v, 6), classes_of(rows, v, 7)
    loss, lse, dloss = torch.empty(rows, device="cuda"), torch.full((rows,), 6.0, device="cuda"), torch.rand(rows, device="cuda")
    bias, dbias, dw = torch.zeros(v, device="cuda"), torch.empty(v, device="cuda"), torch.empty_like(w)
    random = words(3, 4)
    return [
        (api.LayerNormForward(h, x, y, residual=r, total=t), dict(x=x, gamma=vec, y=y, beta=vec2, residual=r, total=t), ("y", "total")),
        (api.LayerNormBackward(h, dy, r, dx, dtotal=x), dict(dy=dy, total=r, gamma=vec, dx=dx, dgamma=dg, dbeta=db, dtotal=x),
         ("dx", "dgamma", "dbeta")),
        (api.DropoutForward(h, x, y, p=0.3, residual=r), dict(x=x, random=random, y=y, residual=r), ("y",)),
        (api.DropoutBackward(h, dy, dx, p=0.3), dict(dy=dy, random=random, dx=dx), ("dx",)),
        (api.EmbeddingForward(h, tokens, table, y), dict(tokens=tokens, table=table, y=y), ("y",)),
        (api.EmbeddingBackward(h, tokens, dy, dtable), dict(tokens=tokens, dy=dy, dtable=dtable), ("dtable",)),
        (api.CrossEntropyForward(h, x, w, target), dict(x=x, w=w, target=target, loss=loss, lse=lse.clone(), bias=bias), ("loss", "lse")),
        (api.CrossEntropyBackward(h, x, w, target, dx, dw),
         dict(x=x, w=w, target=target, lse=lse, dloss=dloss, dx=dx, dw=dw, bias=bias, dbias=dbias), ("dx", "dw", "dbias"))]


def wrong(t):
    if t.dim() == 2:
        yield "fewer rows", t[:-1]
        yield "another type", t.to(F32 if t.dtype == BF else BF)
        yield "transposed", t.t().contiguous().t()
        yield "other strides", torch.cat([t, t], 1)[:, :t.shape[1]]
    else:
        yield "shorter", t[1:]
        yield "apart", torch.stack([t, t], 1)[:, 0]
        yield "another type", t.to(torch.int32 if t.dtype == torch.int64 else torch.float64)
    yield "on the host", t.cpu()


def test_tensors_unlike_their_examples_are_refused(handle):
    for op, right, _ in calls(handle):
        op(**right)
        before = handle.launches()
        for name, t in right.items():
            for what, bad in wrong(t):
                with pytest.raises(ValueError, match=name):
                    op(**{**right, name: bad})
                    pytest.fail(f"{type(op).__name__} took {name} {what}")
        assert handle.launches() == before
        op(**right)
    handle.synchronize()


def test_closed_operators_are_refused(handle):
    for op, right, _ in calls(handle):
        op(**right)
        op.close()
        before = handle.launches()
        with pytest.raises(B.DlcError) as e:
            op(**right)
        assert e.value.status in (B.DLC_STATUS_BAD_PARAM, B.DLC_STATUS_NOT_INITIALIZED)
        assert handle.launches() == before


def test_wrong_arguments_are_refused(handle):
    x, y = rand(20, 64, dtype=BF), torch.empty(20, 64, dtype=BF, device="cuda")
    for p in (-0.1, 1.0, 1.5, float("nan")):
        with pytest.raises(ValueError):
            api.DropoutForward(handle, x, y, p=p)
    tokens, table = tokens_of(20, 30, 1), rand(30, 64, dtype=BF)
    for bad in (tokens[:-1], tokens.repeat(2), tokens.cpu(), torch.stack([tokens, tokens], 1)[:, 0]):
        with pytest.raises(ValueError):
            api.EmbeddingForward(handle, bad, table, y)
        with pytest.raises(ValueError):
            api.CrossEntropyForward(handle, x, table, bad)
    with pytest.raises(TypeError):
        api.EmbeddingForward(handle, tokens.short(), table, y)
    for scale in (float("inf"), float("nan"), 1e39):
        with pytest.raises(B.DlcError):
            api.EmbeddingForward(handle, tokens, table, y, scale=scale)(tokens, table, y)
    with pytest.raises(B.DlcError):  # channels that do not match
        api.EmbeddingForward(handle, tokens, rand(30, 32, dtype=BF), y)(tokens, rand(30, 32, dtype=BF), y)
    with pytest.raises(B.DlcError):  # FP32 operands of the product
        api.CrossEntropyForward(handle, x.float(), table.float(), tokens)
    with pytest.raises(B.DlcError):  # no gradient wanted
        api.CrossEntropyBackward(handle, x, table, tokens)(x, table, tokens, torch.ones(20, device="cuda"), torch.ones(20, device="cuda"))
    f8 = torch.float8_e4m3fn
    loss, lse = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    with pytest.raises(B.DlcError):  # E4M3 without scales
        api.CrossEntropyForward(handle, x.to(f8), table.to(f8), tokens)(x.to(f8), table.to(f8), tokens, loss, lse)
    with pytest.raises(B.DlcError):  # no gradient of E4M3
        api.CrossEntropyBackward(handle, x.to(f8), table.to(f8), tokens, y)
    scale = torch.empty(20, device="cuda")
    with pytest.raises(B.DlcError):  # a scale with a BF16 output
        api.LayerNormForward(handle, x, y)(x, torch.ones(64, device="cuda"), y, scale=scale)
    with pytest.raises(B.DlcError):
        api.LayerNormForward(handle, x, y, eps=-1.0)(x, torch.ones(64, device="cuda"), y)
    handle.synchronize()


def test_indices_beyond_32_bits_are_refused(handle):
    """Rows of almost 2^31 channels, and tables of as many rows."""
    c = 2 ** 31 - 1
    x, y = torch.empty(1, c, dtype=BF, device="cuda"), torch.empty(1, c, dtype=BF, device="cuda")
    gamma, token, state = torch.empty(c, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    long, thin = torch.empty(c, 1, dtype=BF, device="cuda"), torch.empty(1, 1, dtype=BF, device="cuda")
    before = handle.launches()
    for call in (lambda: api.LayerNormForward(handle, x, y)(x, gamma, y),
                 lambda: api.LayerNormBackward(handle, x, x, y)(x, x, gamma, y),
                 lambda: api.DropoutForward(handle, x, y, p=0.5)(x, state, y),
                 lambda: api.EmbeddingForward(handle, token, x, y)(token, x, y),
                 lambda: api.EmbeddingForward(handle, token, long, thin)(token, long, thin),
                 lambda: api.EmbeddingBackward(handle, token, x, y),
                 lambda: api.EmbeddingBackward(handle, token, thin, long),
                 lambda: api.CrossEntropyForward(handle, x, x, token),
                 lambda: api.CrossEntropyForward(handle, thin, long, token),
                 lambda: api.CrossEntropyBackward(handle, thin, long, token)):
        with pytest.raises(B.DlcError) as e:
            call()
        assert e.value.status == B.DLC_STATUS_NOT_SUPPORTED
    assert handle.launches() == before


def test_outputs_over_inputs_are_refused(handle):
    rows, c, v = 40, 64, 40
    buf = rand(rows + 1, c, dtype=BF)
    x, shifted = buf[:rows], buf[1:]
    g = torch.ones(c, device="cuda")
    tokens, vec = tokens_of(rows, v, 1), torch.empty(rows, device="cuda")
    other = torch.empty_like(x)
    tries = [
        (api.LayerNormForward(handle, x, shifted), (x, g, shifted)),
        (api.LayerNormBackward(handle, x, other, shifted), (x, other, g, shifted)),
        (api.DropoutForward(handle, x, shifted, p=0.1), (x, words(1, 2), shifted)),
        (api.DropoutBackward(handle, x, shifted, p=0.1), (x, words(1, 2), shifted)),
        (api.EmbeddingForward(handle, tokens, x, shifted), (tokens, x, shifted)),
        (api.EmbeddingBackward(handle, tokens, x, shifted), (tokens, x, shifted)),
        (api.CrossEntropyForward(handle, x, x, tokens), (x, x, tokens, vec, vec)),
        (api.CrossEntropyBackward(handle, x, other, tokens, shifted), (x, other, tokens, vec, vec, shifted))]
    before = handle.launches()
    for op, args in tries:
        with pytest.raises(B.DlcError) as e:
            op(*args)
        assert e.value.status == B.DLC_STATUS_BAD_PARAM, type(op).__name__
    assert handle.launches() == before


@pytest.mark.parametrize("rows,c,v", [(40, 60, 33), (90, 72, 70), (300, 128, 513)])
def test_neighbours_of_outputs_are_left_alone(handle, rows, c, v):
    """Outputs in the middle of wider buffers: what lies beside and behind them stays."""
    def inside(n, ch):
        big = torch.full((n + 2, ch + 24), 7.0, dtype=BF, device="cuda")
        return big, big[1:n + 1, 8:8 + ch]

    def vector(n):
        big = torch.full((n + 16,), 7.0, device="cuda")
        return big, big[8:8 + n]

    def table(n, ch):
        big = torch.full((n + 2, ch), 7.0, dtype=BF, device="cuda")
        return big, big[1:n + 1]

    x, r, dy = (rand(rows, c, seed=i, dtype=BF) for i in (1, 2, 3))
    w, tokens, target = rand(v, c, seed=4, dtype=BF), tokens_of(rows, v, 5), classes_of(rows, v, 6)
    g, lse0, dloss = torch.ones(c, device="cuda"), torch.full((rows,), 6.0, device="cuda"), torch.rand(rows, device="cuda")
    (b1, y), (b2, t), (b3, dx) = inside(rows, c), inside(rows, c), inside(rows, c)
    (b4, dg), (b5, db), (b6, loss), (b7, lse), (b8, dbias) = vector(c), vector(c), vector(rows), vector(rows), vector(v)
    (b9, dtable), (b10, dw) = table(v, c), table(v, c)

    def check(*pairs):
        for big, part in pairs:
            rest = big.clone()
            at = (part.data_ptr() - big.data_ptr()) // big.element_size()
            rest.as_strided(part.shape, part.stride(), at).fill_(7.0)
            assert (rest == 7.0).all()
            assert torch.isfinite(part.float()).all()
            big.fill_(7.0)

    api.LayerNormForward(handle, x, y, residual=r, total=t)(x, g, y, residual=r, total=t)
    check((b1, y), (b2, t))
    api.LayerNormBackward(handle, dy, r, dx)(dy, r, g, dx, dgamma=dg, dbeta=db)
    check((b3, dx), (b4, dg), (b5, db))
    api.DropoutForward(handle, x, y, p=0.5)(x, words(1, 1), y)
    check((b1, y))
    api.EmbeddingForward(handle, tokens, w, y)(tokens, w, y)
    check((b1, y))
    api.EmbeddingBackward(handle, tokens, dy, dtable)(tokens, dy, dtable)
    check((b9, dtable))
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse)
    check((b6, loss), (b7, lse))
    api.CrossEntropyBackward(handle, x, w, target, dx, dw)(x, w, target, lse0, dloss, dx, dw, dbias=dbias)
    check((b3, dx), (b10, dw), (b8, dbias))


@pytest.mark.parametrize("rows", [24, 300, 5000])
def test_replayed_graphs_follow_their_inputs(rows):
    """Every operator captured once; replays on new values in the same tensors give what
    eager calls give, also after other calls have used the operators' workspaces."""
    s = torch.cuda.Stream()
    with api.Handle(s) as h, torch.cuda.stream(s):
        ops = calls(h, rows=rows)
        for op, right, _ in ops:
            op(**right)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            h.set_stream(torch.cuda.current_stream())
            for op, right, _ in ops:
                op(**right)
        h.set_stream(s)
        inputs = ("x", "dy", "residual", "w", "table")
        for turn in range(3):
            for op, right, outs in ops:
                for name in inputs:
                    if name in right and name not in outs:
                        right[name].copy_(rand(*right[name].shape, seed=10 * turn + len(name), dtype=BF))
            graph.replay()
            s.synchronize()
            # the operators share output tensors: only the last writer's values are looked at
            seen, want = {}, []
            for op, right, outs in ops:
                for name in outs:
                    seen[right[name].data_ptr()] = (op, right, name, right[name].clone())
            for op, right, outs in ops:
                op(**right)
                s.synchronize()
                for name in outs:
                    last = seen[right[name].data_ptr()]
                    if last[0] is op:
                        want.append((type(op).__name__, name, last[3], right[name].clone()))
            assert len(want) >= 8
            for kind, name, got, eager in want:
                assert torch.equal(got, eager), (kind, name, turn)


def test_operators_on_another_stream_than_their_tensors(handle):
    """Work queued on the handle's stream waits for nothing else; ordered by an event, it
    sees what the current stream wrote."""
    s = torch.cuda.Stream()
    with api.Handle(s) as h:
        for op, right, outs in calls(h, rows=600):
            torch.cuda.synchronize()
            op(**right)
            s.synchronize()
            want = [right[n].clone() for n in outs]
            for n in outs:
                right[n].fill_(float("nan"))
            s.wait_stream(torch.cuda.current_stream())
            op(**right)
            torch.cuda.current_stream().wait_stream(s)
            for n, w in zip(outs, want):
                assert torch.equal(right[n], w), (type(op).__name__, n)


def test_embedding_of_a_table_of_more_than_2_31_elements(handle):
    v, c, rows = 1100000, 2048, 70
    table = torch.empty(v, c, dtype=BF, device="cuda")
    tokens = torch.randint(v - 50, v, (rows,), generator=torch.Generator().manual_seed(1)).cuda()
    tokens[:5] = torch.tensor([0, 1, v - 1, 524288 * 2, -1])
    table[tokens[tokens >= 0]] = rand(int((tokens >= 0).sum()), c, seed=2, dtype=BF)
    y = torch.empty(rows, c, dtype=BF, device="cuda")
    api.EmbeddingForward(handle, tokens, table, y)(tokens, table, y)
    assert torch.equal(y, torch.where((tokens >= 0)[:, None], table[tokens.clamp(min=0)], 0.0))
    api.EmbeddingBackward(handle, tokens, y, table)(tokens, y, table)
    named = tokens[tokens >= 0].unique()
    places = torch.searchsorted(named, tokens.clamp(min=0))
    want, err = ref.embedding_backward(torch.where(tokens >= 0, places, -1), d(y), named.numel(), 1.0)
    close(table[named], want, err + cref.stored(want, BF), "dtable")
    table[named] = 0
    assert not table.any()


@pytest.mark.parametrize("rows", [20, 70])
def test_cross_entropy_of_weights_of_more_than_2_31_elements(handle, rows):
    v, c = 1100000, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(v, c, dtype=BF, device="cuda").normal_(0, c ** -0.5, generator=g)
    x, target = rand(rows, c, seed=2, dtype=BF), classes_of(rows, v, 3)
    target[:3] = torch.tensor([v - 1, 1048600, 0])
    loss, lse, dloss = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.rand(rows, device="cuda")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse)
    f = ref.cross_entropy(d(x), d(w), target)
    close(lse, *f["lse"], "lse")
    close(loss, *f["loss"], "loss")
    dw = torch.empty_like(w)
    api.CrossEntropyBackward(handle, x, w, target, None, dw)(x, w, target, lse, dloss, dw=dw)
    _, (want, err), _ = ref.cross_entropy_backward(d(x), d(w), target, f, d(dloss), BF, BF)
    del f
    close(dw, want, err, "dw")


@pytest.mark.parametrize("rows,c,v", [(1, 257, 3), (40, 1001, 70), (3, 300, 1), (300, 2047, 40)])
@pytest.mark.parametrize("shift", [0, 1, 2, 5, 7])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_operands_at_any_address_are_copied_whole(handle, rows, c, v, shift, pad):
    """A product whose operands begin anywhere in a 16-byte piece, between values that are none, is that of
    aligned ones."""
    def placed(t, pitch):
        n = t.shape[0] * pitch
        out = torch.full((n + 16,), float("nan"), dtype=BF, device="cuda")[shift:shift + n].view(t.shape[0], pitch)[:, :t.shape[1]]
        out.copy_(t)
        return out
    wide = (c + 15) // 16 * 16
    x, w = rand(rows, c, seed=1, dtype=BF), rand(v, c, seed=2, dtype=BF)
    aligned = [torch.nn.functional.pad(t, (0, wide - c)) for t in (x, w)]
    y, want = torch.empty(rows, v, device="cuda"), torch.empty(rows, v, device="cuda")
    xs, ws = placed(x, c + pad), placed(w, c)
    api.LinearForward(handle, xs, ws, y)(xs, ws, y)
    api.LinearForward(handle, *aligned, want)(*aligned, want)
    # sums of c products in FP32 in some order each: c / 2 roundings of a sum of size sum |x w| at most
    bound = 2.0 ** -24 * c * (x.double().abs() @ w.double().abs().T)
    assert ((y.double() - want.double()).abs() <= bound).all()
