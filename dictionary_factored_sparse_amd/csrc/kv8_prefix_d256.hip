// kv8_prefix_d256.hip -- kv8_prefix_attention for head_dim 256.
#include "kv8_prefix_kernel.hpp"

template void dfs::launch_prefix<256>(const PrefixLaunch&, const PrefixWs&, const PrefixCut&, hipStream_t);
