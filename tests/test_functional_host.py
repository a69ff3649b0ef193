"""CPU tests of the autograd forms: what they hand to the library, with the
library's calls replaced by recorders."""
import pytest
import torch

from optimizer_step_dl_amd import _abi, functional

F32 = torch.float32


@pytest.fixture
def default_dtype(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


@pytest.mark.parametrize("default_dtype", [torch.float64, torch.bfloat16, torch.float16, F32], indirect=True)
def test_losses_under_any_default_dtype(default_dtype, monkeypatch):
    """Totals, losses, log-probabilities, records and default weights are
    FP32, whatever torch's default is."""
    seen = []

    def record(logits, *args, **kw):
        values = [a for a in (*args, *kw.values()) if torch.is_tensor(a) and a.is_floating_point()]
        seen.append([v.dtype for v in values if v is not kw.get("grad")])
        for v in values:
            v.zero_()

    monkeypatch.setattr(_abi, "radamw_policy_loss", record)
    monkeypatch.setattr(_abi, "radamw_preference_loss", record)
    monkeypatch.setattr(_abi, "radamw_logits_grad", lambda logits, labels, stats, grad, upstream: seen.append(
        [stats.dtype, upstream.dtype]))
    x = torch.zeros((6, 5), dtype=F32, requires_grad=True)
    labels = torch.tensor([0, 1, -100, 4, 2, 3])
    total, loss, logp = functional.policy_loss(x, labels, torch.zeros(6))
    total.backward()
    assert total.dtype == loss.dtype == logp.dtype == F32
    total, loss, seq = functional.preference_loss(x, labels, torch.tensor([0, 2, 6]), torch.zeros(2))
    total.backward()
    assert total.dtype == loss.dtype == seq.dtype == F32
    # advantages, total, loss, logp, weights, records; the records and the upstream value;
    # the reference's sums, total, loss, seq_logp, logp, records, weights; the same two
    assert [len(d) for d in seen] == [6, 2, 7, 2]
    assert all(d == F32 for call in seen for d in call), seen


class Streams:
    """Stands in for torch.cuda's streams and events: current_stream() hands
    out the given names in turn, everything submitted is written down."""

    def __init__(self, names):
        self.names, self.log, self.events = iter(names), [], 0

    def current_stream(self, device=None):
        self.name = next(self.names)
        return self

    def wait_event(self, event):
        self.log.append((self.name, "waits for", event.of))

    def event(self):
        owner = self

        class Event:
            def record(self, stream):
                self.of = f"write {owner.events}"
                owner.events += 1
                owner.log.append((stream.name, "records", self.of))

        return Event()


def test_grad_buffer_is_written_in_order(monkeypatch):
    """Two uses of a table with one buffer, whose forward passes ran on two
    streams: the second write waits for the first, and the table's own
    gradient node and the stream that called backward() for both."""
    s = Streams(["A", "B", "node", "node", "caller", "caller"])
    monkeypatch.setattr(torch.cuda, "current_stream", s.current_stream)
    monkeypatch.setattr(torch.cuda, "Event", s.event)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(_abi, "_raw_stream", None)
    monkeypatch.setattr(functional, "_buffer_writes", {}, raising=False)
    monkeypatch.setattr(_abi, "radamw_embedding_lookup", lambda table, ids, out, scale: out.zero_())
    monkeypatch.setattr(_abi, "radamw_embedding_grad_workspace_bytes", lambda n, rows, dim: 0)
    monkeypatch.setattr(_abi, "radamw_embedding_grad", lambda *a: s.log.append("writes"))
    table = torch.zeros((5, 4), requires_grad=True)
    buffer = torch.zeros((5, 4))
    ids = torch.tensor([1, 2])
    x, y = (functional.embedding(ids, table, grad_buffer=buffer) for _ in range(2))
    (x.sum() + y.sum()).backward()
    first, second = "write 0", "write 1"
    assert s.log == ["writes", ("A", "records", first), ("B", "waits for", first), "writes", ("B", "records", second),
                     ("node", "waits for", first), ("node", "waits for", second),
                     ("caller", "waits for", first), ("caller", "waits for", second)]
    assert table.grad is None


def test_grad_buffer_refused_write_leaves_no_trace(monkeypatch):
    """Under capture nothing is waited for (the library refuses the call), and
    a refused write is no write that others wait for."""
    s = Streams(["A"])
    monkeypatch.setattr(torch.cuda, "current_stream", s.current_stream)
    monkeypatch.setattr(torch.cuda, "Event", s.event)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(functional, "_buffer_writes", {None: s.event()}, raising=False)
    monkeypatch.setattr(_abi, "radamw_embedding_lookup", lambda table, ids, out, scale: out.zero_())
    monkeypatch.setattr(_abi, "radamw_embedding_grad_workspace_bytes", lambda n, rows, dim: 0)

    def refuse(*a):
        raise _abi.RadamwError(-1, "radamw_embedding_grad")

    monkeypatch.setattr(_abi, "radamw_embedding_grad", refuse)
    table = torch.zeros((5, 4), requires_grad=True)
    x = functional.embedding(torch.tensor([1, 2]), table, grad_buffer=torch.zeros((5, 4)))
    with pytest.raises(_abi.RadamwError):
        x.sum().backward()
    assert s.log == []
