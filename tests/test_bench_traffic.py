"""The benchmark's DRAM traffic is read from a committed capture, keyed to the source of the
kernel that it was taken of: a change of the kernel needs a new capture."""


def test_the_captures_are_of_the_present_kernels():
    import json
    import os
    import bench
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        for key, t in json.load(f).items():
            assert bench.committed_traffic(key, t["workload"]) == t["dram_bytes_read"] + t["dram_bytes_write"], key
