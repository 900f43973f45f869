"""Plans from several host threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_plans_of_different_sizes_from_two_threads():
    """Batches whose offsets take different amounts of shared memory, each on its own stream."""
    import block_sparse_attention_nsa_gb300 as nsa
    go, errors, sets = threading.Barrier(2), [], []
    for b in (3600, 16384):
        lens = torch.arange(b, dtype=torch.int32, device="cuda") % 7
        table = torch.arange(b, dtype=torch.int32, device="cuda").view(b, 1)
        want = (torch.repeat_interleave(table.view(-1), lens.long()) * 8
                + torch.cat([torch.arange(int(n), device="cuda") for n in lens[:7]]).repeat(b // 7 + 1)[
                    :int(lens.sum())]).int()
        sets.append((b, lens, table, torch.zeros_like(lens), want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(b, lens, table, start, want, stream):
        try:
            with torch.cuda.stream(stream):
                slots, cu = torch.empty_like(want), torch.empty(b + 1, dtype=torch.int32, device="cuda")
                go.wait(60)
                for _ in range(20000):
                    nsa.page_slots(table, start, lens, 8, b, slots, cu)
                stream.synchronize()
                assert torch.equal(slots, want) and int(cu[-1].item()) == want.numel()
        except Exception as e:      # noqa: BLE001 -- handed to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
