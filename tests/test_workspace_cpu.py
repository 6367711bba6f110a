"""The binding's workspaces, with host memory in the place of the device's:
which buffer a call gets, and which ones stay."""
import threading
import types

import pytest
import torch

import exact_lloyd_means_flashassign_amd as fk

DEV = torch.device("cuda", 0)


@pytest.fixture
def card(monkeypatch):
    """A card whose current stream and recording state the test sets."""
    state = types.SimpleNamespace(stream=7, recording=False)
    empty = torch.empty

    def host(*shape, **kw):
        kw.pop("device", None)
        return empty(*shape, **kw)
    monkeypatch.setattr(torch, "empty", host)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=state.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.recording)
    monkeypatch.setattr(fk, "_raw_stream", lambda d: state.stream)
    fk._ws_cache.clear()
    yield state
    fk._ws_cache.clear()


def calls():
    return (lambda n: fk._workspace(n, DEV), lambda n: fk._scratch(n, 0, None))


@pytest.mark.parametrize("i", (0, 1))
def test_a_stream_keeps_its_buffer(card, i):
    get = calls()[i]
    p, n = get(5000)[:2]
    assert p % 256 == 0 and n >= 5000
    assert get(400)[:2] == (p, n)
    card.stream = 8
    assert get(400)[0] != p
    card.stream = 7
    assert get(400)[:2] == (p, n)


@pytest.mark.parametrize("i", (0, 1))
def test_a_recorded_call_has_a_buffer_of_its_own(card, i):
    """The graph holds the buffer's address, so neither may a later call of the
    stream share it nor may its growth free it."""
    get = calls()[i]
    before = get(5000)
    card.recording = True
    first, second = get(400), get(9000)
    card.recording = False
    assert first[0] % 256 == 0 and first[1] >= 400 and second[1] >= 9000
    assert len({before[0], first[0], second[0]}) == 3
    # the stream has its buffer still, and what it grows to is none of theirs
    assert get(5000)[:2] == before[:2]
    grown = get(20000)
    assert grown[1] >= 20000 and grown[0] not in (first[0], second[0])
    assert get(400)[:2] == grown[:2]


def test_a_given_workspace_is_taken_as_it_is(card, monkeypatch):
    mine = torch.empty(4096, dtype=torch.uint8)
    monkeypatch.setattr(fk, "_dev", lambda t, *a: t)
    for card.recording in (False, True):
        assert fk._workspace(100, DEV, mine)[:2] == (mine.data_ptr(), 4096)
        assert fk._scratch(100, 0, mine)[:2] == (mine.data_ptr(), 4096)
    assert not fk._ws_cache


@pytest.mark.parametrize("i", (0, 1))
def test_threads_of_one_stream_have_buffers_of_their_own(card, i):
    """A call's kernels may be enqueued between those of another thread's call."""
    get = calls()[i]
    mine = get(5000)
    theirs = []
    t = threading.Thread(target=lambda: theirs.extend((get(5000), get(300))))
    t.start()
    t.join()
    assert theirs[0][0] == theirs[1][0] != mine[0]
    assert get(300)[:2] == mine[:2]


class OnCard(torch.Tensor):
    """A host tensor that says it lies on a card (nothing here reaches one)."""
    card = 0
    is_cuda = True

    def get_device(self):
        return self.card


def on_card(card, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnCard)
    t.card = card
    return t


def test_a_workspace_of_another_card_is_refused(monkeypatch):
    """Every other argument on card 0, the workspace on card 1."""
    def launched(*a):
        raise AssertionError("the call went on to its launch")
    monkeypatch.setattr(fk, "_run", launched)
    ws = on_card(1, 1 << 20, dtype=torch.uint8)
    X, W, one = on_card(0, 4, 8), on_card(0, 6, 8), on_card(0, 4)
    for call in (lambda: fk.fk_layer_norm_backward(X, X, one, one, dX=on_card(0, 4, 8), workspace=ws),
                 lambda: fk.fk_route(X, 2, workspace=ws),
                 lambda: fk.fk_linear(X, W, workspace=ws),
                 lambda: fk.fk_linear_backward(on_card(0, 4, 6), X, W, workspace=ws)):
        with pytest.raises(ValueError, match="different devices"):
            call()
