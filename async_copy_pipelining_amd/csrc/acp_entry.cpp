// The entry points of the library in one translation unit: they share the
// calling thread's error reason and launch text, the descriptor checks and
// the device attributes of acp_api.cpp.
#include "acp_api.cpp"
#include "acp_rows_api.hpp"
#include "acp_heads_api.hpp"
#include "acp_attn_api.hpp"
