"""The lengths of bench.py's serving case, without a GPU."""
import bench


def test_serve_lengths_span_half_to_all_of_the_stated_context():
    assert bench.serve_lengths(1, 1000) == [1000]        # one request: of the stated length
    assert bench.serve_lengths(2, 1001) == [1001, 500]
    n = bench.serve_lengths(32, 8192)
    assert len(n) == 32 and n[0] == max(n) == 8192 and n[-1] == min(n) == 4096 and len(set(n)) == 32
