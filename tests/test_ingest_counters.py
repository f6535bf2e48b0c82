"""bench.py --ingest-counters takes one run's counters and refuses a folder
that holds those of several: an older run's file would be stored as if it were
measured on the current sources."""
import pytest

import bench

HEAD = "Dispatch_Id,Kernel_Name,Counter_Name,Counter_Value\n"


def _run(folder, name, counter, kib):
    """Two markers' groups of one M (3 launches of kib KiB each) and the calibration copy of 512 MiB."""
    mark, own, copy = "at::FillFunctor<int>", "hm::k_any", "copy_kernel"
    rows = [mark] + [own] * 3 + [mark] + [copy]
    text = "".join(f"{i},{n},{counter},{512 * 1024 if n is copy else kib}\n" for i, n in enumerate(rows))
    (folder / name).write_text(HEAD + text)


def test_one_run_a_folder(tmp_path):
    dirs = []
    for counter in ("FETCH_SIZE", "WRITE_SIZE"):
        d = tmp_path / counter / "host"
        d.mkdir(parents=True)
        _run(d, "11_counter_collection.csv", counter, 100)
        dirs.append(tmp_path / counter)
    got = bench.ingest_counters(*map(str, dirs))
    assert got["FETCH_SIZE"]["per_group"] == [100 * 1024] and got["WRITE_SIZE"]["calib"] == 1.0
    _run(dirs[0] / "host", "12_counter_collection.csv", "FETCH_SIZE", 200)
    with pytest.raises(ValueError, match="one counter file"):
        bench.ingest_counters(*map(str, dirs))
    with pytest.raises(ValueError, match="one counter file"):
        bench.ingest_counters(str(tmp_path / "none"), str(dirs[1]))
