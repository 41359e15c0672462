"""What the kernels' sources must not hold."""
import pathlib

CSRC = pathlib.Path(__file__).parent.parent / "video_dit_long_gb300" / "csrc"


def test_every_tile_copy_lands_in_one_cta():
    """The kernels also run as one rank of several GPUs (bench.py --gpus N), where copies that land in several CTAs and
    clusters of CTAs that share them are ruled out: each CTA loads its own tiles."""
    found = 0
    for f in sorted(CSRC.iterdir()):
        text = f.read_text()
        found += text.count("cp.async.bulk.tensor")
        for word in ("multicast", "mapa.shared", "barrier.cluster", "cudaLaunchAttributeClusterDimension", "__cluster_dims__"):
            assert word not in text.lower() and word not in text, (f.name, word)
    assert found  # the copies are in these files


def test_the_traffic_record_is_of_the_present_kernel():
    """bench.py reports null traffic once the attention kernel's code differs from the captured one's: an edit of its
    sources, the shared device header among them, needs a new capture in profiles/traffic.txt."""
    import bench
    for workload in ("pro_n8", "long_n16"):
        assert bench.traffic_record(bench.STEP_KERNEL, workload), (workload, bench.source_digest(bench.STEP_KERNEL))
