"""The DRAM traffic that bench.py reports is of the kernels as they are."""
import bench
import synth


def test_traffic_is_that_of_the_sources():
    assert bench.NCU_TRAFFIC["sources_sha256"] == bench.kernel_sources_sha256()
    specs = bench.all_workload_specs()
    for name, total in bench.NCU_TRAFFIC["bytes"].items():
        step = synth.make_step(specs[name], with_accept=False)
        least = bench.verify_algorithmic_bytes(specs[name], step.seq_lens)
        # every page once, and the split partials written and read back
        assert least < total < 1.05 * least, name
        assert bench.ncu_traffic(name) == total
