// kv8_prefix_d128.hip -- kv8_prefix_attention for head_dim 128.
#include "kv8_prefix_kernel.hpp"

template void dfs::launch_prefix<128>(const PrefixLaunch&, const PrefixWs&, const PrefixCut&, hipStream_t);
