// library.hip - the translation unit of the grouped products together with the one function
// by which the other sources set the calling thread's error text: that text
// (mgg_last_error) is private to grouped_gemm.hip.

#include "grouped_gemm.hip"

extern "C" __attribute__((visibility("hidden"))) void mgg_set_last_error(const char* text) {
  g_last_error = text;
}
