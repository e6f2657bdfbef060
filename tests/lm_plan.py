"""Builds and runs tests/lm_plan_probe.cpp: what the feed-forward products' planner chooses."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build(tmp):
    exe = os.path.join(str(tmp), "lm_plan_probe")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", "-isystem", "/opt/rocm/include", "-I",
                           os.path.join(ROOT, "layer_rnn_forward_amd", "csrc"),
                           os.path.join(ROOT, "tests", "lm_plan_probe.cpp"), "-o", exe])
    return exe


def rows(exe, *args):
    out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]
