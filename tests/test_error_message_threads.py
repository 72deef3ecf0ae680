"""Messages of failed context-free calls: every thread reads its own."""
import threading

import pytest

from test_abi import built_lib  # noqa: F401
from text_embedding_encoder_gb300 import binding


def test_a_thread_reads_the_message_of_its_own_failed_call(built_lib):  # noqa: F811
    assert built_lib.tee_layernorm_backward_workspace(-1, 8) == binding.TEE_EINVAL

    def other():
        assert built_lib.tee_embed_backward_workspace(-1, 5, 8) == binding.TEE_EINVAL
        seen.append(built_lib.tee_last_error(None).decode())
    seen = []
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert "embed_backward_workspace" in seen[0]
    assert "layernorm_backward_workspace" in built_lib.tee_last_error(None).decode()


def test_failing_calls_in_many_threads_at_once(built_lib):  # noqa: F811
    """Messages of different lengths, written and read at the same time."""
    calls = [("layernorm_backward", (-1, 8)), ("embed_backward", (-1, 5, 8)), ("vocab_loss_forward", (-1, 5, 8)),
             ("vocab_loss_backward", (5, 0, 8))]
    wrong = []
    start = threading.Barrier(8)

    def run(k):
        name, sizes = calls[k % len(calls)]
        start.wait()
        for _ in range(2000):
            try:
                binding.workspace_bytes(name, *sizes)
            except binding.TeeError as e:
                if name + "_workspace" not in str(e):
                    wrong.append((name, str(e)))
            else:
                wrong.append((name, "no error"))
    threads = [threading.Thread(target=run, args=(k,)) for k in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


def test_no_message_in_a_thread_without_a_failed_call(built_lib):  # noqa: F811
    with pytest.raises(binding.TeeError):
        binding.workspace_bytes("embed_backward", -1, 5, 8)
    seen = []
    t = threading.Thread(target=lambda: seen.append(built_lib.tee_last_error(None).decode()))
    t.start()
    t.join()
    assert seen == [""]
