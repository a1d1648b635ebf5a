"""bf16 layer calls that take the GPU alone (64 experts and more, or experts served by both
tile shapes) run beside no other bf16 layer's, whatever streams they are queued on.
Streams and events are stand-ins and the launches left out, so nothing here needs a
device; what is checked is the order that the queues are left with."""
import contextlib
import threading

import pytest
import torch

BF = torch.bfloat16
D, E, K, F = 64, 64, 2, 128
DEFAULT, A, B, EXT = 0, 11, 12, 99  # handles; EXT: a stream that torch does not keep


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


class World:
    """Queues of (what, ...) by stream handle, and which streams are being captured."""

    def __init__(self):
        self.queues, self.capturing, self.current, self.inside = {}, set(), [DEFAULT], 0

    def put(self, key, *what):
        self.queues.setdefault(key, []).append(what)

    def before(self, key, n):
        """The launches that entry n of the queue comes behind."""
        seen, todo, done = set(), [(key, n)], {}
        while todo:
            key, n = todo.pop()
            if done.get(key, 0) >= n:
                continue
            for what in self.queues[key][done.get(key, 0):n]:
                if what[0] == "launch":
                    seen.add(what[1])
                else:
                    todo.append(what[1])
            done[key] = n
        return seen


@pytest.fixture
def world(monkeypatch):
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe
    w = World()

    class Stream:
        def __init__(self, key):
            self.key = self.cuda_stream = key
            self.stream_id = key if key == EXT else 3

        def record_event(self):
            assert self.key not in w.capturing
            return (self.key, len(w.queues.get(self.key, [])))

        def wait_event(self, event):
            assert self.key not in w.capturing
            w.put(self.key, "wait", event)

        def wait_stream(self, other):
            self.wait_event(other.record_event())

    @contextlib.contextmanager
    def stream(s):
        w.current.append(s.key)
        yield
        w.current.pop()
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: Stream(DEFAULT))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(w.current[-1]))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.current[-1] in w.capturing)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw).as_subclass(OnDevice))
    monkeypatch.setattr(moe, "_stream", lambda s: w.current[-1] if s is None else
                        s if isinstance(s, int) else s.cuda_stream)
    monkeypatch.setattr(moe, "_turns", type(moe._turns)(moe._turns.default_factory))
    monkeypatch.setattr(moe, "_version", lambda x: 0)

    def launch(name):
        def fn(cfg, *a, stream=None):
            w.inside += 1
            assert w.inside == 1  # one host thread at a time
            w.put(stream, "launch", len([q for qs in w.queues.values() for q in qs if q[0] == "launch"]))
            w.inside -= 1
            if name == "fails":
                raise RuntimeError("refused")
        return fn
    for name in ("moe_forward", "moe_backward"):
        monkeypatch.setattr(moe, name, launch(name))
    w.moe, w.launch, w.Stream, w.monkeypatch = moe, launch, Stream, monkeypatch
    return w


def layer(w, dtype=BF, E=E):
    def zeros(*shape, dtype=dtype):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    return w.moe.MoELayer(zeros(E, D, dtype=torch.float32), zeros(E, D, 2 * F), zeros(E, F, D), K)


def rows(n=16, dtype=BF):
    return torch.zeros(n, D, dtype=dtype).as_subclass(OnDevice)


def latest(w, key):
    """The launches that the queue's last launch comes behind."""
    q = w.queues[key]
    n = max(i for i, what in enumerate(q) if what[0] == "launch")
    return q[n][1], w.before(key, n)


def test_calls_follow_one_another(world):
    w, lay, x, out = world, layer(world), rows(), rows()
    for key in (A, A, B, DEFAULT, A, EXT, EXT, B):
        lay.forward(x, out, stream=w.Stream(key))
        n, behind = latest(w, key)
        assert behind == set(range(n))
        lay.backward(x, out, stream=w.Stream(key))
        n, behind = latest(w, key)
        assert behind == set(range(n))


def test_two_layers_and_the_current_stream(world):
    w, one, two, x = world, layer(world), layer(world), rows()
    one(x, rows(), stream=A)
    with torch.cuda.stream(w.Stream(B)):
        two(x, rows())
    assert latest(w, B) == (1, {0})
    two(x, rows(), stream=EXT)
    one(x, rows())
    assert latest(w, DEFAULT) == (3, {0, 1, 2})


def test_one_stream_waits_for_nothing(world):
    w, lay, x = world, layer(world), rows()
    for _ in range(3):
        lay(x, rows())
    assert [q[0] for q in w.queues[DEFAULT]] == ["launch"] * 3


def test_fp32_layers_run_side_by_side(world):
    w, lay, x = world, layer(world, torch.float32), rows(dtype=torch.float32)
    for key in (A, B, A):
        lay(x, rows(dtype=torch.float32), stream=w.Stream(key))
    assert all(q[0] == "launch" for qs in w.queues.values() for q in qs)


def test_a_stream_that_is_gone_is_not_touched(world):
    """Its event was recorded when its call was launched."""
    w, lay, x = world, layer(world), rows()
    lay(x, rows(), stream=EXT)
    seen = len(w.queues[EXT])
    w.monkeypatch.setattr(torch.cuda, "ExternalStream", lambda key: pytest.fail("gone") if key == EXT else w.Stream(key))
    lay(x, rows(), stream=A)
    assert w.queues[A][0] == ("wait", (EXT, seen))


@pytest.mark.parametrize("key", [A, EXT])
def test_captured_calls_wait_for_nothing(world, key):
    w, lay, x = world, layer(world), rows()
    lay(x, rows(), stream=B)
    w.capturing.add(key)
    with torch.cuda.stream(w.Stream(key)):
        lay(x, rows())
    w.capturing.clear()
    assert [q[0] for q in w.queues[key]] == ["launch"]
    lay(x, rows(), stream=DEFAULT)  # ... and the next eager call still follows the first
    assert 0 in latest(w, DEFAULT)[1]
    # a capture on the stream of the latest call, and a call elsewhere in the meantime
    lay(x, rows(), stream=w.Stream(key))
    w.capturing.add(key)
    if key == EXT:
        lay(x, rows(), stream=B)  # by the event of that call
        assert latest(w, B)[1] >= {0, 2, 3}
    else:
        with pytest.raises(RuntimeError, match="captured"):
            lay(x, rows(), stream=B)
        w.capturing.clear()
        lay(x, rows(), stream=B)


def test_a_call_that_fails_counts(world):
    """Some of its kernels may run."""
    w, lay, x = world, layer(world), rows()
    w.monkeypatch.setattr(w.moe, "moe_forward", w.launch("fails"))
    with pytest.raises(RuntimeError, match="refused"):
        lay(x, rows(), stream=A)
    w.monkeypatch.setattr(w.moe, "moe_forward", w.launch("moe_forward"))
    lay(x, rows(), stream=B)
    assert latest(w, B) == (1, {0})


def test_host_threads(world):
    w, x = world, rows()
    layers, errors = [layer(w) for _ in range(4)], []

    def run(lay, key):
        try:
            for _ in range(50):
                lay.forward(x, rows(), stream=w.Stream(key))
        except BaseException as e:
            errors.append(e)
    threads = [threading.Thread(target=run, args=(lay, 20 + i)) for i, lay in enumerate(layers)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    order = {q[1]: (key, i) for key, qs in w.queues.items() for i, q in enumerate(qs) if q[0] == "launch"}
    assert sorted(order) == list(range(200))
    for n in range(1, 200):
        key, i = order[n]
        assert n - 1 in w.before(key, i)


def test_which_calls_run_alone(world):
    alone = world.moe._alone
    for T, E, k, want in ((16, 64, 2, True), (4096, 256, 8, True), (255, 8, 2, False), (256, 8, 2, True),
                          (2047, 8, 2, True), (2048, 8, 2, False), (4096, 8, 2, False), (64, 16, 4, False)):
        assert alone(world.moe.config(T, D, E, k, F)) == want, (T, E, k)


def test_other_calls_run_beside_one_another(world):
    w, small, x = world, layer(world, E=8), rows()
    for key in (A, B, A, DEFAULT, B):
        small(x, rows(), stream=w.Stream(key))
    assert all(q[0] == "launch" for qs in w.queues.values() for q in qs)


def test_other_calls_run_beside_none_that_runs_alone(world):
    w, small, lay, x = world, layer(world, E=8), layer(world), rows()
    small(x, rows(), stream=w.Stream(A))  # 0, 1: beside one another
    small(x, rows(), stream=EXT)
    lay(x, rows(), stream=w.Stream(B))    # 2: behind both
    assert latest(w, B) == (2, {0, 1})
    small(x, rows(), stream=w.Stream(A))  # 3, 4: behind 2, beside one another
    small(x, rows(), stream=EXT)
    assert latest(w, A) == (3, {0, 1, 2}) and latest(w, EXT) == (4, {0, 1, 2})
    small(x, rows(), stream=w.Stream(A))  # no second wait
    assert [q[0] for q in w.queues[A]] == ["launch", "wait", "launch", "launch"]
    small(x, rows(), stream=w.Stream(B))  # 6: on the stream of 2
    lay(x, rows(), stream=DEFAULT)        # 7: behind all
    assert latest(w, DEFAULT) == (7, set(range(7)))


def test_streams_that_come_and_go_are_forgotten(world):
    """... by a call now and then that follows all of them."""
    w, small, x = world, layer(world, E=8), rows()
    w.monkeypatch.setattr(w.moe._Turns, "keeps", lambda self, stream, key: False)
    for i in range(1000):
        small(x, rows(), stream=1000 + i)
        assert len(w.moe._turns[0].ends) <= w.moe._MOST_STREAMS
    lay = layer(w)
    lay(x, rows(), stream=A)
    assert latest(w, A) == (1000, set(range(1000)))
