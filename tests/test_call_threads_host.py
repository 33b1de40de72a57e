"""The first calls of two threads at once (no GPU work): whatever one has done so
far, the other's call goes through."""
import sys
import threading

import pytest

from selective_state_space_mamba_amd import _call


class Tensor:
    """What launch_stream asks of one."""
    is_cuda = True
    device = "cuda:0"

    def get_device(self):
        return 0


@pytest.fixture
def fresh(monkeypatch):
    """launch_stream as in a new process, with its two sources standing in for torch's."""
    monkeypatch.setattr(_call, "_raw_current", lambda: lambda dev: 7 + dev)
    monkeypatch.setattr(_call, "_device", lambda: lambda: 0)

    def reset():
        for name in list(vars(_call)):
            if name in ("_torch_calls", "_current", "_current_device"):
                monkeypatch.setattr(_call, name, None)

    return reset


def test_a_second_thread_between_any_two_steps_of_the_first(fresh):
    """Another thread makes a whole call before each instruction of the first one's, one instruction a run."""
    code = _call.launch_stream.__code__
    at, runs = 0, 0
    while True:
        fresh()
        seen, other, failed = 0, [], []

        def second():
            try:
                other.append(_call.launch_stream(Tensor(), None))
            except Exception as e:  # noqa: BLE001
                failed.append(e)

        def trace(frame, event, arg):
            nonlocal seen
            if frame.f_code is not code:
                return None
            frame.f_trace_opcodes = True
            if event == "opcode":
                if seen == at:
                    t = threading.Thread(target=second)
                    t.start()
                    t.join()
                seen += 1
            return trace

        old = sys.gettrace()
        sys.settrace(trace)
        try:
            first = _call.launch_stream(Tensor(), None)
        finally:
            sys.settrace(old)
        if at >= seen:
            break
        assert not failed and first == 7 and other == [7], (at, failed)
        at, runs = at + 1, runs + 1
    assert runs > 20
