// kv8_prefix_d64.hip -- kv8_prefix_attention for head_dim 64.
#include "kv8_prefix_kernel.hpp"

template void dfs::launch_prefix<64>(const PrefixLaunch&, const PrefixWs&, const PrefixCut&, hipStream_t);
