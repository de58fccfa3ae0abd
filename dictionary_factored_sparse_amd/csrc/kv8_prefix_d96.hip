// kv8_prefix_d96.hip -- kv8_prefix_attention for head_dim 96.
#include "kv8_prefix_kernel.hpp"

template void dfs::launch_prefix<96>(const PrefixLaunch&, const PrefixWs&, const PrefixCut&, hipStream_t);
