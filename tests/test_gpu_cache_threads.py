"""fd_build_tables from two host threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fd():
    import decode_attention_decoding_gb300 as fd
    return fd


def test_two_threads_build_tables_of_large_batches(fd):
    """Batches whose lengths want more than 48 KB of shared memory, of two sizes, on two streams: no
    call may lower what the other one's launch needs.  Every request gets one token and one page."""
    calls, failed, wrong = 3000, [], []
    start = threading.Barrier(2)

    def work(batch):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            one = torch.ones(batch, dtype=torch.int32, device="cuda")
            free = torch.arange(batch, dtype=torch.int32, device="cuda")
            count = torch.full((1,), batch, dtype=torch.int32, device="cuda")
            table = torch.full((batch, 2), -1, dtype=torch.int32, device="cuda")
            stream.synchronize()
            start.wait()
            for _ in range(calls):
                try:
                    t = fd.fd_build_tables(torch.zeros_like(one), one, table, free, count, 16, batch, batch)
                except fd.FdError as e:
                    failed.append((batch, str(e)))
                    return
            stream.synchronize()
            if not torch.equal(t.slot_map, torch.arange(batch - 1, -1, -1, device="cuda") * 16) or int(t.free_count) != 0:
                wrong.append(batch)

    threads = [threading.Thread(target=work, args=(b,)) for b in (4096, 3100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong, (failed, wrong)
