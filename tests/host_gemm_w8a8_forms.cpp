// The choice of the W8A8 linear layer's form (gemm_w8a8_forms.hpp) for tests/test_gemm_w8a8_forms.py: the form's number, and
// 16 more for rows at any address.
#include "../quantized_state_space_amd/csrc/gemm_w8a8_forms.hpp"

extern "C" int host_form(int64_t M, int64_t N, int64_t K, int yf16, int direct) {
  const qssm::FormChoice c = qssm::choose_form(M, N, K, yf16 != 0, direct != 0);
  return c.form + (c.shift ? 16 : 0);
}
