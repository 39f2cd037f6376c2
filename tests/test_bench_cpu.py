"""bench.py's host side: the counter summary it reports traffic from goes with
the kernel sources it was taken on."""
import bench


def test_the_default_workload_reports_its_traffic():
    t = bench.load_traffic(bench.kernel_source_sha(), "hyena-d1024-l16k", "closed-loop tanh")
    assert t is not None
