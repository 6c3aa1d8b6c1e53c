// overlap() of common.hpp for the host, on arrays of cases (tests/test_host_overlap.py).
#include "../quantized_state_space_amd/csrc/common.hpp"

// c: n rows of (address, rows, stride, width) of the one tensor and of the other; out: 1 where they overlap
extern "C" void host_overlap(const int64_t* c, int64_t n, uint8_t* out) {
  for (int64_t i = 0; i < n; ++i, c += 8) {
    const qssm::Span a{(const void*)(uintptr_t)c[0], c[1], c[2], c[3]}, b{(const void*)(uintptr_t)c[4], c[5], c[6], c[7]};
    out[i] = qssm::overlap(a, b);
  }
}
