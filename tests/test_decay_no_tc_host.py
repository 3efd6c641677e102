"""bf16 sequences of the decayed attention where the library is built without its tensor-core path: refused (CPU)."""
import os
import subprocess

from video_diffusion_linear_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_bf16_without_the_tensor_core_path_is_refused(tmp_path):
    obj = os.path.join(build.PKG, "_build", "decay.o")
    build.build(force=not os.path.exists(obj))
    exe = tmp_path / "decay_no_tc"
    subprocess.run([build.NVCC, "-std=c++17", "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC,
                    "-x", "cu", *build.ARCH, "-c", os.path.join(HERE, "c", "decay_no_tc_check.cpp"), "-o", str(tmp_path / "m.o")],
                   check=True)
    subprocess.run([build.NVCC, *build.ARCH, "-o", str(exe), str(tmp_path / "m.o"), obj], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert out[:5] == ["forward 2", "backward 2", "bf16 sizes 0 0", "f32 sizes 1 1", "launches 0"]
